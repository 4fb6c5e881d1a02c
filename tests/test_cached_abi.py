"""Incremental scoring without a GPU: the oracle's pins, the turning rates and
the refusals of every argument the host can judge."""
import ctypes

import numpy as np
import pytest

import classifier_scoring_b200 as rm
from classifier_scoring_b200 import build
from oracle import cached as C


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


# --- the oracle's own pins ---------------------------------------------------------

def test_oracle_slots_worked_example():
    # page of 4; request 0 holds 3 tokens in page 9 and gets 2: one fits page 9, one opens page 5
    table = np.array([[9, 0], [0, 0], [7, 8]], dtype=np.int32)
    off, pos, slot, after, used, bad, tab = C.kv_slots([3, 0, 8], [2, 0, 1], 4, [5, 6], 0, table, 4)
    assert off.tolist() == [0, 2, 2, 2] and bad == 1       # request 2 would need a third page of its row
    assert pos.tolist() == [3, 4, 0, 0] and slot.tolist() == [39, 20, -1, -1]
    assert after.tolist() == [5, 0, 8] and used == 1 and tab.tolist() == [[9, 5], [0, 0], [7, 8]]


def test_oracle_rotation_keeps_relative_positions():
    # <rot(q, m), rot(k, n)> depends on m - n alone, in both layouts
    r = np.random.RandomState(0)
    q, k = r.randn(1, 1, 16), r.randn(1, 1, 16)
    f = C.rope_freqs(16, 100.0)
    for layout in (0, 1):
        dots = [(C.norm_rope(q, None, 0, [m], f, layout)[0] * C.norm_rope(k, None, 0, [m - 7], f, layout)[0]).sum()
                for m in (7, 50, 1000)]
        assert np.allclose(dots, dots[0], rtol=0, atol=1e-9)


def test_oracle_window_of_everything_is_causal_attention():
    r = np.random.RandomState(1)
    q, k, v = r.randn(9, 2, 8), r.randn(9, 1, 8), r.randn(9, 1, 8)
    full = C.attend_window(q, k, v, [0, 9], 0, 0)[0]
    assert np.array_equal(full, C.attend_window(q, k, v, [0, 9], 9, 0)[0])
    assert np.allclose(full, C.attend_window(q, k, v, [0, 9], 3, 9)[0], atol=1e-15)   # sinks cover the rest
    one = C.attend_window(q, k, v, [0, 9], 1, 0)[0]
    assert np.allclose(one, np.repeat(v, 2, axis=1), atol=1e-15)                      # itself alone


# --- turning rates -----------------------------------------------------------------

@pytest.mark.parametrize("name,scaling", [("plain", 0), ("linear", 1), ("base", 2), ("parts", 3)])
@pytest.mark.parametrize("rot,base,factor", [(128, 10000.0, 8.0), (64, 5e5, 1.0), (36, 100.0, 3.5), (4, 10.0, 2.0)])
def test_rope_freqs(name, scaling, rot, base, factor):
    got = rm.ops.rope_freqs(rot, base, scaling, factor, trained=2048, fast=32, slow=1)
    ref = C.rope_freqs(rot, base, name, factor, trained=2048, fast=32, slow=1)
    assert np.allclose(got, ref, rtol=1e-13, atol=0)
    if name == "parts" and factor > 1 and rot == 128:
        assert got[0] == 1.0 and np.isclose(got[-1], ref[-1]) and got[-1] < C.rope_freqs(rot, base)[-1] / 7.9


@pytest.mark.parametrize("kw", [dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=258), dict(base=1.0), dict(base=float("nan")),
                                dict(scaling=4), dict(scaling=1, factor=0.5), dict(scaling=1, factor=float("inf")),
                                dict(scaling=2, rot_dim=2, factor=2.0), dict(scaling=3, factor=2.0, trained=0.0),
                                dict(scaling=3, factor=2.0, trained=10.0, fast=1.0, slow=1.0),
                                dict(scaling=3, factor=2.0, trained=10.0, fast=1.0, slow=0.0)])
def test_rope_freqs_refuses(kw):
    with pytest.raises(rm.RmError) as e:
        rm.ops.rope_freqs(**{"rot_dim": 64, **kw})
    assert e.value.code == rm.RM_E_INVAL


# --- refusals ----------------------------------------------------------------------
# Every pointer is a made-up 16-byte aligned address: the host refuses the call before it looks at memory.
A = 1 << 20


def cache(**kw):
    a = dict(k=A, v=A, n_pages=10, page_size=16, n_kv_heads=2, head_dim=64, dtype=rm.BF16)
    a.update(kw)
    return rm.KvCache(a.pop("k"), a.pop("v"), **a)


def refused(call, code=None):
    with pytest.raises(rm.RmError) as e:
        call()
    assert e.value.code == (rm.RM_E_INVAL if code is None else code)
    assert str(e.value)


SLOTS = dict(len_before=A, n_new=A, n_seqs=4, page_size=16, free_pages=A, n_free=8, used_before=A, block_table=A,
             table_stride=4, T=8, offsets=A, positions=A, slots=A, len_after=A, used_after=A, unserved=A)


@pytest.mark.parametrize("kw", [{k: None} for k, v in SLOTS.items() if v == A]
                         + [dict(n_seqs=0), dict(page_size=0), dict(page_size=1025), dict(n_free=-1),
                            dict(table_stride=0), dict(T=-1)])
def test_slots_refuses(kw):
    refused(lambda: rm.ops.kv_slots(**{**SLOTS, **kw}))


def test_slots_refuses_too_many_sequences():
    refused(lambda: rm.ops.kv_slots(**{**SLOTS, "n_seqs": 16385}), rm.RM_E_RANGE)


ROPE = dict(qkv=A, qkv_stride=384, q_out=A, q_stride=128, k_out=A, k_stride=128, T=5, n_q_heads=2, n_kv_heads=2,
            head_dim=64, q_gain=A, k_gain=A, eps=1e-6, positions=A, slots=A)


@pytest.mark.parametrize("kw", [dict(qkv=None), dict(q_out=None), dict(T=-1), dict(n_q_heads=3), dict(n_q_heads=0),
                                dict(n_kv_heads=0), dict(head_dim=60), dict(head_dim=264), dict(head_dim=0),
                                dict(qkv_stride=376), dict(qkv_stride=388), dict(q_stride=120), dict(k_stride=64),
                                dict(qkv=A + 8), dict(q_out=A + 2), dict(k_out=A + 8), dict(q_gain=None),
                                dict(eps=-1.0), dict(eps=float("nan")), dict(positions=None), dict(slots=None),
                                dict(rope=rm.Rope(None, 64)), dict(rope=rm.Rope(A, 63)), dict(rope=rm.Rope(A, 66)),
                                dict(rope=rm.Rope(A, -2)), dict(rope=rm.Rope(A, 64, layout=2)),
                                dict(cache=cache(n_kv_heads=1)), dict(cache=cache(head_dim=128)),
                                dict(cache=cache(k=None)), dict(cache=cache(dtype=rm.F32)),
                                dict(cache=cache(page_size=0)), dict(cache=cache(n_pages=0)),
                                dict(cache=cache(page_stride=2 * 16 * 64 - 8)), dict(cache=cache(page_stride=2 * 16 * 64 + 4)),
                                dict(cache=cache(page_stride=1 << 62)), dict(cache=cache(v=A + 8)),
                                dict(cache=cache(k_scale=A)), dict(cache=cache(k_scale=A, v_scale=A)),
                                dict(cache=cache(dtype=rm.E4M3, v_scale=A))])
def test_qk_norm_rope_refuses(kw):
    refused(lambda: rm.ops.qk_norm_rope(**{**ROPE, "rope": rm.Rope(A, 64), "cache": cache(), **kw}))


@pytest.mark.parametrize("kw", [dict(q_gain=A + 2), dict(k_gain=A + 1), dict(q_gain=A + 6, k_gain=A + 4)])
def test_qk_norm_rope_refuses_gains_that_no_float_lies_at(kw):
    refused(lambda: rm.ops.qk_norm_rope(**{**ROPE, "rope": rm.Rope(A, 64), "cache": cache(), **kw}))


WINDOW = dict(q=A, q_stride=128, k=A, k_stride=128, v=A, v_stride=128, offsets_dev=A, n_seqs=1, T=5, n_q_heads=2,
              n_kv_heads=2, head_dim=64, window=0, sinks=0, out=A, out_stride=128)


@pytest.mark.parametrize("kw", [{k: None} for k, v in WINDOW.items() if v == A]
                         + [dict(n_seqs=0), dict(T=-1), dict(n_q_heads=3), dict(n_kv_heads=0), dict(head_dim=32),
                            dict(window=-1), dict(sinks=-1), dict(q_stride=64), dict(k_stride=132), dict(out_stride=0),
                            dict(q=A + 2), dict(out=A + 8), dict(n_q_heads=129, n_kv_heads=1, q_stride=1 << 14, out_stride=1 << 14)])
def test_attn_window_refuses(kw):
    refused(lambda: rm.ops.attn_window(**{**WINDOW, **kw}))


def test_steps_of_no_tokens_take_empty_buffers():
    # an empty tensor has no address
    rope = dict(qkv=None, q_out=None, k_out=None, T=0, positions=None, slots=None)
    for more in ({}, dict(rope=None), dict(cache=None), dict(q_gain=None, k_gain=None)):
        rm.ops.qk_norm_rope(**{**ROPE, "rope": rm.Rope(A, 64), "cache": cache(), **rope, **more})
    rm.ops.attn_window(**{**WINDOW, "q": None, "k": None, "v": None, "out": None, "T": 0})
    for kw in (dict(q_stride=64), dict(offsets_dev=None), dict(head_dim=32)):      # the rest is judged as ever
        refused(lambda: rm.ops.attn_window(**{**WINDOW, "T": 0, **kw}))
    refused(lambda: rm.ops.qk_norm_rope(**{**ROPE, **rope, "rope": rm.Rope(None, 64)}))


DECODE = dict(q=A, q_stride=128, block_table=A, table_stride=4, length=A, n_seqs=3, n_q_heads=2, window=0, sinks=0, out=A,
              out_stride=128, workspace=A, workspace_bytes=1 << 30)


@pytest.mark.parametrize("kw", [{k: None} for k, v in DECODE.items() if v == A]
                         + [dict(n_seqs=0), dict(table_stride=0), dict(n_q_heads=3), dict(window=-1), dict(sinks=-1),
                            dict(q_stride=64), dict(out_stride=132), dict(q=A + 2), dict(out=A + 8), dict(workspace=A + 8),
                            dict(cache=cache(head_dim=32)), dict(cache=cache(k=None)), dict(cache=cache(page_size=2000))])
def test_attn_decode_refuses(kw):
    refused(lambda: rm.ops.attn_decode(**{**DECODE, "cache": cache(), **kw}))


def test_attn_decode_refuses_a_small_workspace():
    refused(lambda: rm.ops.attn_decode(**{**DECODE, "cache": cache(), "workspace_bytes": 0}), rm.RM_E_RANGE)


def test_decode_workspace_size():
    size = rm.ops.attn_decode_workspace(4, 2, cache())
    assert size > 0
    for bad in (lambda: rm.ops.attn_decode_workspace(0, 2, cache()), lambda: rm.ops.attn_decode_workspace(4, 3, cache()),
                lambda: rm.ops.attn_decode_workspace(4, 2, cache(head_dim=8))):
        refused(bad)


def test_without_a_device_the_calls_say_so():
    import torch
    if torch.cuda.is_available():
        pytest.skip("there is a device")
    for call in (lambda: rm.ops.kv_slots(**SLOTS), lambda: rm.ops.attn_window(**WINDOW),
                 lambda: rm.ops.attn_decode(**DECODE, cache=cache()),
                 lambda: rm.ops.qk_norm_rope(**ROPE, rope=rm.Rope(A, 64), cache=cache())):
        refused(call, rm.RM_E_DEVICE)


def test_timeouts_refuse_and_say_when_there_is_no_device():
    import torch
    assert rm.lib().rm_op_timeouts(None) == rm.RM_E_INVAL
    for limit in (0, 999, 10 ** 10 + 1, -5):
        refused(lambda: rm.selftest_op_wait(limit))
    if not torch.cuda.is_available():
        refused(rm.op_timeouts, rm.RM_E_CUDA)


class Buffer:
    """What the binding asks of a tensor: its device (-1: host) and its address."""

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device

    def data_ptr(self):
        return A


@pytest.mark.parametrize("call", [
    lambda x: rm.KvCache(Buffer(1), x, n_pages=4, page_size=16, n_kv_heads=1, head_dim=64),
    lambda x: rm.ops.kv_slots(**{**SLOTS, "offsets": Buffer(1), "free_pages": x}),
    lambda x: rm.ops.attn_window(**{**WINDOW, "out": Buffer(1), "offsets_dev": x}),
    lambda x: rm.ops.attn_decode(**{**DECODE, "q": Buffer(1), "length": x, "cache": cache()}),
    lambda x: rm.ops.qk_norm_rope(**{**ROPE, "qkv": Buffer(1), "positions": x}, rope=rm.Rope(A, 64), cache=cache())])
@pytest.mark.parametrize("where", ["host", "numpy", "another device"])
def test_buffers_that_are_not_on_the_calls_device_are_refused(call, where):
    x = {"host": Buffer(-1), "numpy": np.zeros(64), "another device": Buffer(0)}[where]
    refused(lambda: call(x))


def test_a_cache_or_rotation_of_another_device_is_refused():
    for host in (Buffer(-1), np.zeros(32)):
        refused(lambda: rm.Rope(host, 64))
    other = cache(k=Buffer(0), v=Buffer(0))
    refused(lambda: rm.ops.attn_decode(**{**DECODE, "q": Buffer(1), "cache": other}))
    refused(lambda: rm.ops.qk_norm_rope(**{**ROPE, "qkv": Buffer(1)}, rope=rm.Rope(A, 64), cache=other))
    refused(lambda: rm.ops.qk_norm_rope(**{**ROPE, "qkv": Buffer(1)}, rope=rm.Rope(Buffer(0), 64), cache=cache()))


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(rm.KvCache(A, A, n_pages=1, page_size=1, n_kv_heads=1, head_dim=8)._args) == 64
    assert ctypes.sizeof(rm.Rope(A, 2)._args) == 24
