"""What the 8-bit cache, attention weights and eviction refuse, each refusal by its own reason, without
a GPU.  Nothing here launches."""

import contextlib

import pytest
import torch

from paged_kv_cache_exact_b200 import api
from paged_kv_cache_exact_b200 import binding as B
from test_cache_cpu import ATTN, ATTN_OK, BF, W_TAIL, _append, _call, _evict, _q8, _tensors, _weights

MOST = 65535 * 128                          # keys of a prompt's weights: a grid's second axis of 128-key tiles


@pytest.mark.parametrize("kw", [dict(q_len=300), dict(q_len=2, S=40)], ids=["rows", "scores too many for the split kernel"])
def test_a_prompts_weights_over_too_many_keys_are_refused_before_the_attention_runs(kw):
    kw = dict(kw, max_len=MOST + 1, stride=MOST + 1, maxp=1 << 20)
    assert _call("paged_attn_weights", ATTN + W_TAIL[0], ATTN_OK + W_TAIL[1], kw) == B.PKV_ERR_UNSUPPORTED
    # one key fewer is not refused for its size: the workspace is asked for
    kw.update(max_len=MOST, stride=MOST, ws=None)
    assert _call("paged_attn_weights", ATTN + W_TAIL[0], ATTN_OK + W_TAIL[1], kw) == B.PKV_ERR_WORKSPACE


@pytest.mark.parametrize("q_len,off", [(300, 0), (300, 2 * 8 * 300 * 256 - 16), (300, -16), (17, 0)])
def test_prompt_weights_with_an_output_over_q_are_refused(q_len, off):
    """A prompt's weights read q again after out is written."""
    q = 1 << 24
    kw = dict(q=q, out=q + off, q_len=q_len)
    assert _call("paged_attn_weights", ATTN + W_TAIL[0], ATTN_OK + W_TAIL[1], kw) == B.PKV_ERR_INVALID_ARG


# -------------------------------------------------------- the tensor-level functions' own checks --


class Reached(Exception):
    """The checks of shapes and types let the call through to the check of devices."""


@pytest.fixture
def no_devices(monkeypatch):
    def stop(*tensors):
        raise Reached
    monkeypatch.setattr(api, "_on_device", stop)


def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


I32, I64, F64, HALF = torch.int32, torch.int64, torch.float64, torch.float16
POOL, SCALES, ROWS = "of one type", r"scales must be \[pages", r"k_new and v_new must be"
WEIGHTS, TABLES = r"weights must be float32 \[num_seqs", "hold a row"


@pytest.mark.parametrize("f", [_q8, _weights, _evict, _append])
def test_tensors_that_fit_pass_every_check_of_shapes(no_devices, f):
    with pytest.raises(Reached):
        f()


@pytest.mark.parametrize("f,kw,why", [
    (_q8, dict(q=z(2, 8, 1, 128)), "q must be bf16"),
    (_q8, dict(q=z(2, 8, 128, dtype=torch.bfloat16)), "q must be bf16"),
    (_weights, dict(q=z(2, 8, 1, 128, dtype=HALF)), "q must be bf16"),
    (_q8, dict(q=z(2, 8, 1, 64, dtype=torch.bfloat16)), "q's head dim"),
    (_q8, dict(k=z(8, 16, 4, 128, dtype=torch.int8)), POOL),
    (_q8, dict(v=z(8, 32, 4, 128, dtype=torch.uint8)), POOL),
    (_evict, dict(v=z(8, 32, 2, 128, dtype=torch.int8)), POOL),
    (_append, dict(k=z(8, 32, 512, dtype=torch.int8), v=z(8, 32, 512, dtype=torch.int8)), POOL),
    (_q8, dict(ks=None), "needs its scales"), (_evict, dict(vs=None), "needs its scales"),
    (_q8, dict(ks=z(8, 3, 4)), SCALES), (_q8, dict(ks=z(8, 2, 2)), SCALES), (_append, dict(vs=z(7, 2, 4)), SCALES),
    (_weights, dict(ks=z(8, 0, 4), vs=z(8, 0, 4)), SCALES), (_evict, dict(ks=z(8, 8), vs=z(8, 8)), SCALES),
    (_q8, dict(vs=z(8, 2, 4, dtype=F64)), "scales must be float32"),
    (_append, dict(ks=z(8, 2, 4, dtype=HALF)), "scales must be float32"),
    (_weights, dict(k=BF, v=BF), "only an 8-bit cache has scales"),
    (_evict, dict(k=BF, v=BF), "only an 8-bit cache has scales"),
    (_q8, dict(table=z(2, 4, dtype=I64)), "must be int32"), (_weights, dict(lens=z(2, dtype=I64)), "must be int32"),
    (_evict, dict(lens=z(2, dtype=I64)), "must be int32"), (_evict, dict(dst=z(2, 4, dtype=I64)), "must be int32"),
    (_append, dict(cu=z(3, dtype=I64)), "must be int32"),
    (_q8, dict(lens=z(3, dtype=I32)), TABLES), (_q8, dict(table=z(8, dtype=I32)), TABLES),
    (_weights, dict(table=z(3, 4, dtype=I32)), TABLES),
    (_evict, dict(dst=z(2, 5, dtype=I32)), TABLES), (_evict, dict(table=z(3, 4, dtype=I32)), TABLES),
    (_weights, dict(w=z(2, 4, 99)), WEIGHTS), (_weights, dict(w=z(2, 8, 100)), WEIGHTS),
    (_weights, dict(w=z(2, 4, 100, dtype=F64)), WEIGHTS), (_weights, dict(w=z(8, 100)), WEIGHTS),
    (_evict, dict(w=z(2, 4, 50)), WEIGHTS), (_evict, dict(w=z(2, 4, 100, dtype=F64)), WEIGHTS),
    (_append, dict(new=z(3, 2, 128)), ROWS), (_append, dict(new=z(3, 512)), ROWS),
    (_append, dict(cu=z(2, dtype=I32)), r"num_seqs \+ 1 entries"),
    (_append, dict(table=z(3, 4, dtype=I32)), "a row for each"),
])
def test_each_value_error_has_its_own_reason(no_devices, f, kw, why):
    with pytest.raises(ValueError, match=why):
        f(**kw)


@pytest.mark.parametrize("q_len,dtype", [(2, torch.bfloat16), (1, torch.float32)])
def test_an_output_that_is_not_like_q(no_devices, q_len, dtype):
    t = _tensors()
    with pytest.raises(ValueError, match="out must look like q"):
        api.paged_q8(t["q"], t["k"], t["v"], t["ks"], t["vs"], t["table"], t["lens"], 32, True, 0.1, 100,
                     out=z(2, 8, q_len, 128, dtype=dtype))


def test_other_pairs_that_do_not_match(no_devices):
    t = _tensors()
    with pytest.raises(ValueError, match="page_size"):
        api.paged_q8(t["q"], t["k"], t["v"], t["ks"], t["vs"], t["table"], t["lens"], 16, True, 0.1, 100)
    with pytest.raises(ValueError, match=WEIGHTS):
        api.evict(t["k"], t["v"], t["w"], t["table"], t["lens"], 16, 4, 100, weights_out=z(2, 4, 101),
                  k_scales=t["ks"], v_scales=t["vs"])
    with pytest.raises(ValueError, match="as many sources"):
        api.copy_pages_q8(t["k"], t["v"], t["ks"], t["vs"], z(2, dtype=I32), z(3, dtype=I32))
    with pytest.raises(ValueError, match="must be int32"):
        api.copy_pages_q8(t["k"], t["v"], t["ks"], t["vs"], z(2, dtype=I64), z(2, dtype=I64))


@pytest.mark.parametrize("f,kw", [
    (_q8, dict(k=BF, v=BF, ks=None, vs=None)), (_append, dict(k=BF, v=BF, ks=None, vs=None)),
    (_evict, dict(k=BF.half(), v=BF.half(), ks=None, vs=None)),
    (_weights, dict(k=BF.half(), v=BF.half(), ks=None, vs=None)),
])
def test_caches_of_another_type_are_type_errors(no_devices, f, kw):
    with pytest.raises(TypeError, match="unsupported cache dtype"):
        f(**kw)


def test_rows_of_another_type_are_a_type_error(monkeypatch):
    monkeypatch.setattr(api, "_on_device", lambda *t: contextlib.nullcontext())
    monkeypatch.setattr(api, "_stream_of", lambda stream, t: 0)
    monkeypatch.setattr(B, "paged_kv_append_q8", lambda *a: pytest.fail("launched"))
    with pytest.raises(TypeError, match="unsupported dtype torch.float16"):
        _append(new=z(3, 4, 128, dtype=HALF))


class OnDevice:
    def __init__(self, device, contiguous=True):
        self.device, self.contiguous = device, contiguous

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return self.contiguous


@pytest.mark.parametrize("devices,contiguous,why", [
    ((-1, -1), (True, True), "one CUDA device"), ((0, 1), (True, True), "one CUDA device"),
    ((0, -1), (True, True), "one CUDA device"), ((0, 0), (True, False), "must be contiguous"),
    ((1, 1), (False, True), "must be contiguous"),
])
def test_tensors_of_two_devices_or_with_gaps(devices, contiguous, why):
    with pytest.raises(ValueError, match=why):
        api._on_device(*(OnDevice(*x) for x in zip(devices, contiguous)))


def test_a_workspace_with_gaps_or_of_another_device():
    with pytest.raises(ValueError, match="workspace"):
        api._workspace(z(64, dtype=torch.uint8)[::2], 10, torch.device("cpu"))
    with pytest.raises(ValueError, match="workspace"):
        api._workspace(z(64, dtype=torch.uint8), 10, torch.device("meta"))
    assert api._workspace(None, 0, torch.device("cpu")) == (None, 0)
    ws, n = api._workspace(z(64, dtype=torch.float32), 10, torch.device("cpu"))
    assert n == 256
