"""Incremental scoring on the GPU against the fp64 oracle: slot maps, the norm
and rotation with the cache write, windowed attention over packed sequences,
and attention of one new token over the paged cache."""
import numpy as np
import pytest
import torch

import classifier_scoring_b200 as rm
from oracle import cached as C
from tests.helpers import F32_RTOL

pytestmark = pytest.mark.gpu
HALF_BF16 = 2.0 ** -8        # one rounding to bf16, relative
HALF_E4M3 = 2.0 ** -4        # one rounding to e4m3, relative; below 2^-6 its step is 2^-9
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rm.lib()
    torch.cuda.init()


def dev(a, dtype):
    return torch.as_tensor(np.ascontiguousarray(a)).to(dtype).cuda()


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def randn(shape, seed, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def attention_bound(ref, mag, top):
    """P is rounded to bf16 (half a step of each p|v|), the output once more;
    scores and exponentials are fp32, a score's error being relative to its
    sum |q k|, and act on the numerator and on the sum."""
    delta = F32_RTOL * (1 + top[..., None])
    return (HALF_BF16 + 2 * delta + F32_RTOL) * mag + HALF_BF16 * np.abs(ref)


# --- slot maps ----------------------------------------------------------------------

def slots_case(n, lo, hi, far, page, seed, width=None, spare=5, T=None):
    r = np.random.RandomState(seed)
    before, new = r.randint(0, far + 1, n), r.randint(lo, hi + 1, n)
    need = -(-(before + new) // page)
    w = int(need.max()) + 1 if width is None else width
    free = r.permutation(int(need.sum()) + spare).astype(np.int32)
    table = r.randint(0, 1 << 20, (n, w)).astype(np.int32)
    return before, new, free, table, (int(new.sum()) if T is None else T)


def run_slots(before, new, free, table, T, page, used=2, in_place=False, stream=None):
    n = len(before)
    b, m, f, tab = dev(before, torch.int32), dev(new, torch.int32), dev(free, torch.int32), dev(table, torch.int32)
    u = torch.tensor([used], dtype=torch.int32, device="cuda")
    off = torch.full((n + 3,), -7, dtype=torch.int32, device="cuda")
    pos = torch.full((T + 3,), -7, dtype=torch.int32, device="cuda")
    slot = torch.full((T + 3,), -7, dtype=torch.int64, device="cuda")
    after, u2 = (b, u) if in_place else (torch.full_like(b, -7), torch.full_like(u, -7))
    bad = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    rm.ops.kv_slots(b, m, n, page, f, len(free), u, tab, table.shape[1], T, off, pos, slot, after, u2, bad, stream=stream)
    torch.cuda.synchronize()
    assert off[n + 1:].tolist() == [-7, -7] and pos[T:].tolist() == [-7] * 3 and slot[T:].tolist() == [-7] * 3
    return (off[:n + 1].cpu().numpy(), pos[:T].cpu().numpy(), slot[:T].cpu().numpy(), after.cpu().numpy(), int(u2), int(bad),
            tab.cpu().numpy())


def same_slots(got, ref):
    for name, a, b in zip(("offsets", "positions", "slots", "len_after", "used", "unserved", "table"), got, ref):
        assert np.array_equal(a, b), (name, a, b)


@pytest.mark.parametrize("n,lo,hi,far,page", [(1, 1, 1, 0, 1), (1, 0, 0, 9, 4), (5, 0, 3, 40, 16), (64, 1, 1, 4000, 16),
                                              (33, 1, 1, 63, 64), (300, 5, 500, 0, 16), (1025, 0, 7, 1000, 24),
                                              (2, 20000, 30000, 5, 100), (40, 0, 900, 3000, 1024), (4000, 1, 2, 70, 8)])
@pytest.mark.parametrize("in_place", [False, True])
def test_slots(n, lo, hi, far, page, in_place):
    before, new, free, table, T = slots_case(n, lo, hi, far, page, n + hi, spare=7)
    T += 3                                                # a padded batch
    same_slots(run_slots(before, new, free, table, T, page, in_place=in_place),
               C.kv_slots(before, new, page, free, 2, table, T))


@pytest.mark.parametrize("in_place", [False, True])
def test_slots_of_the_most_sequences(in_place):
    before, new, free, table, T = slots_case(16384, 0, 3, 30, 8, 5)
    same_slots(run_slots(before, new, free, table, T, 8, in_place=in_place), C.kv_slots(before, new, 8, free, 2, table, T))


@pytest.mark.parametrize("what", ["pages", "tokens", "row", "negative length", "negative count", "used", "used beyond", "no pages"])
@pytest.mark.parametrize("n", [7, 700, 3000])
def test_slots_serve_what_fits_and_nothing_behind(what, n):
    before, new, free, table, T = slots_case(n, 1, 30, 50, 16, 3 * n)
    used, k = 2, n // 2
    if what == "pages":
        lacking = int((-(-(before + new) // 16) - -(-before // 16)).sum())
        free = free[:2 + lacking // 2]                   # two are in use already
    elif what == "tokens":
        T //= 2
    elif what == "row":
        new[k] += table.shape[1] * 16
    elif what == "negative length":
        before[k] = -1
    elif what == "negative count":
        new[k] = -3
    elif what == "used":
        used = -1
    elif what == "used beyond":
        used = len(free) + 1
    else:
        free = free[:0]
        used = 0
    ref = C.kv_slots(before, new, 16, free, used, table, T)
    assert ref[5] > 0
    same_slots(run_slots(before, new, free, table, T, 16, used=used), ref)
    same_slots(run_slots(before, new, free, table, T, 16, used=used, in_place=True), ref)


def test_slots_of_lengths_near_the_integers_end():
    top = 2 ** 31 - 5
    before, new = np.array([3, top, 4]), np.array([1, 7, 1])
    table = np.zeros((3, 2), dtype=np.int32)
    ref = C.kv_slots(before, new, 1024, np.arange(9), 0, table, 20)
    assert ref[5] == 2
    same_slots(run_slots(before, new, np.arange(9), table, 20, 1024, used=0), ref)


# --- norm, rotation and cache write -----------------------------------------------------

def e4m3_pages(t):
    return f64(t.view(torch.float8_e4m3fn).float())


def rope_case(T, hq, hkv, d, rot, layout, norm, kind, page=16, seed=0, far=5000, mscale=1.0, in_place=False, pad=0,
              bad_slots=(), stream=None):
    hall = hq + 2 * hkv
    qkv = randn((T, hall * d + pad), seed, 1.5)
    r = np.random.RandomState(seed)
    pos = r.randint(0, far + 1, T)
    n_pages = -(-T // page) + 2
    slots = r.permutation(n_pages * page)[:T].astype(np.int64)
    for i, b in bad_slots:
        slots[i] = b if b < 0 else n_pages * page + b
    gains = [1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(seed + k)).cuda() for k in (1, 2)]
    fill = torch.randint(0, 255, (2, n_pages, hkv, page, d + 8), generator=torch.Generator().manual_seed(9), dtype=torch.uint8)
    f8 = kind == "e4m3"
    pages = fill.cuda() if f8 else randn((2, n_pages, hkv, page, d + 8), 7)
    # pages further apart than their content: keys and values of a page beside a gap
    stride = hkv * page * d + 8 * hkv * page
    flat = pages.view(2, n_pages, stride)
    ks = vs = None
    if f8:
        ks, vs = (0.01 + 0.05 * torch.rand(hkv, generator=torch.Generator().manual_seed(seed + k)).cuda() for k in (3, 4))
    cache = rm.KvCache(flat[0], flat[1], n_pages=n_pages, page_size=page, n_kv_heads=hkv, head_dim=d,
                       dtype=rm.E4M3 if f8 else rm.BF16, k_scale=ks, v_scale=vs, page_stride=stride)
    freqs = C.rope_freqs(rot, 10000.0) if rot else np.zeros(1)
    rope = rm.Rope(dev(freqs, torch.float64), rot, layout=layout, mscale=mscale) if rot else None
    x, old = f64(qkv)[:, :hall * d].reshape(T, hall, d), flat.clone()
    before = qkv.clone()
    if in_place:
        q_out, k_out, qs, kst = qkv, qkv[:, hq * d:], hall * d + pad, hall * d + pad
    else:
        q_out = torch.full((T, hq * d + 16), NAN, dtype=torch.bfloat16, device="cuda")
        k_out = torch.full((T, hkv * d + 8), NAN, dtype=torch.bfloat16, device="cuda")
        qs, kst = hq * d + 16, hkv * d + 8
    torch.cuda.synchronize()
    rm.ops.qk_norm_rope(qkv, hall * d + pad, q_out, qs, k_out, kst, T, hq, hkv, d, gains[0] if norm else None,
                        gains[1] if norm else None, 1e-6, rope, dev(pos, torch.int32), cache, dev(slots, torch.int64),
                        stream=stream)
    torch.cuda.synchronize()
    fr = freqs if rot else None
    rq, mq = C.norm_rope(x[:, :hq], f64(gains[0]) if norm else None, 1e-6, pos, fr, layout, mscale)
    rk, mk = C.norm_rope(x[:, hq:hq + hkv], f64(gains[1]) if norm else None, 1e-6, pos, fr, layout, mscale)
    for got, ref, mag, h in ((q_out, rq, mq, hq), (k_out, rk, mk, hkv)):
        g = f64(got)[:, :h * d].reshape(T, h, d)
        assert np.all(np.abs(g - ref) <= HALF_BF16 * np.abs(ref) + 2 * F32_RTOL * mag)
    if in_place:                                            # the value columns and the gap behind them stay
        assert torch.equal(qkv[:, (hq + hkv) * d:], before[:, (hq + hkv) * d:])
    else:
        assert torch.isnan(q_out[:, hq * d:]).all() and torch.isnan(k_out[:, hkv * d:]).all()
        assert torch.equal(qkv, before)
    # the cache: written slots hold the token's heads, everything else is as it was
    v = x[:, hq + hkv:]
    written = np.zeros((n_pages, stride), dtype=bool)
    ok = (slots >= 0) & (slots < n_pages * page)
    for buf, val, mag, scale in ((0, rk, mk, ks), (1, v, np.abs(v), vs)):
        raw = flat[buf]
        vals = e4m3_pages(raw) if f8 else f64(raw)
        for t in np.flatnonzero(ok):
            p, s = divmod(int(slots[t]), page)
            for h in range(hkv):
                a = (h * page + s) * d
                written[p, a:a + d] = True
                g, ref, m = vals[p, a:a + d], val[t, h], mag[t, h]
                if f8:
                    sc = float(scale[h])
                    ref, m = ref / sc, m / sc
                    cut = np.clip(ref, -448, 448)
                    assert np.all(np.abs(g - cut) <= np.maximum(HALF_E4M3 * np.abs(ref), 2.0 ** -10) + 4 * F32_RTOL * m)
                else:
                    assert np.all(np.abs(g - ref) <= HALF_BF16 * np.abs(ref) + 2 * F32_RTOL * m)
        keep = torch.from_numpy(~written).cuda()
        bits = (lambda t: t) if f8 else (lambda t: t.view(torch.int16))
        assert torch.equal(bits(raw)[keep], bits(old[buf])[keep])


@pytest.mark.parametrize("d,rot", [(128, 128), (64, 64), (64, 16), (128, 36), (256, 64), (8, 8), (40, 20), (72, 6), (256, 256), (64, 0),
                                   (96, 96), (200, 2), (16, 12)])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("norm,kind", [(True, "bf16"), (False, "e4m3")])
def test_qk_norm_rope(d, rot, layout, norm, kind):
    rope_case(37, 4, 2, d, rot, layout, norm, kind, seed=d + rot)


@pytest.mark.parametrize("T,hq,hkv", [(1, 1, 1), (1, 16, 16), (3, 10, 2), (129, 12, 12), (700, 5, 1), (65, 33, 3), (2, 128, 1), (33, 64, 8)])
@pytest.mark.parametrize("norm,kind,d", [(True, "e4m3", 64), (False, "bf16", 128), (True, "bf16", 24)])
def test_qk_norm_rope_heads_and_tokens(T, hq, hkv, norm, kind, d):
    rope_case(T, hq, hkv, d, d, 0, norm, kind, page=24, seed=T + hq, mscale=1.25)


@pytest.mark.parametrize("in_place,pad", [(True, 0), (True, 24), (False, 8)])
@pytest.mark.parametrize("d,rot,layout", [(64, 64, 0), (128, 12, 0), (64, 32, 1)])
def test_qk_norm_rope_in_place_and_strides(in_place, pad, d, rot, layout):
    rope_case(50, 6, 3, d, rot, layout, True, "bf16", in_place=in_place, pad=pad, seed=pad)


@pytest.mark.parametrize("d", [24, 64, 128, 256])
@pytest.mark.parametrize("q_at,k_at", [(0, 1), (1, 0), (2, 3), (3, 5), (4, 8)])
def test_qk_norm_rope_gains_anywhere_in_a_parameter_buffer(d, q_at, k_at):
    # gains are fp32 slices of a packed buffer, at any element of it
    T, hq, hkv = 13, 4, 2
    flat = 1 + 0.2 * torch.randn(2 * d + 32, generator=torch.Generator().manual_seed(d)).cuda()
    gq, gk = flat[q_at:q_at + d], flat[d + 8 + k_at:2 * d + 8 + k_at]
    qkv = randn((T, (hq + 2 * hkv) * d), 2)
    outs = []
    for g in ((gq, gk), (gq.clone(), gk.clone())):
        q, k = (torch.full((T, h * d), NAN, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv))
        rm.ops.qk_norm_rope(qkv, (hq + 2 * hkv) * d, q, hq * d, k, hkv * d, T, hq, hkv, d, *g, 1e-6, None, None)
        outs.append((q, k))
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    x = f64(qkv).reshape(T, -1, d)
    for got, rows, g, h in ((outs[0][0], x[:, :hq], gq, hq), (outs[0][1], x[:, hq:hq + hkv], gk, hkv)):
        ref, mag = C.norm_rope(rows, f64(g), 1e-6, None, None, 0)
        assert np.all(np.abs(f64(got).reshape(T, h, d) - ref) <= HALF_BF16 * np.abs(ref) + 2 * F32_RTOL * mag)


def test_qk_norm_rope_far_positions():
    rope_case(64, 4, 2, 128, 128, 0, False, "bf16", far=2 ** 31 - 2, seed=4)


def test_qk_norm_rope_drops_padding_and_bad_slots():
    rope_case(20, 4, 2, 64, 64, 0, True, "bf16", seed=6, bad_slots=((0, -1), (7, 0), (8, 2 ** 40), (19, -2 ** 50)))
    rope_case(20, 4, 2, 64, 64, 1, True, "e4m3", seed=6, bad_slots=((0, -1), (7, 0), (8, 2 ** 40), (19, -2 ** 50)))


def test_qk_norm_rope_without_cache_or_keys():
    qkv = randn((9, 4 * 64), 1)
    q, k = torch.empty(9, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(9, 64, dtype=torch.bfloat16, device="cuda")
    rm.ops.qk_norm_rope(qkv, 256, q, 128, k, 64, 9, 2, 1, 64, None, None, 0.0, None, None)
    torch.cuda.synchronize()
    assert torch.equal(q, qkv[:, :128]) and torch.equal(k, qkv[:, 128:192])     # nothing asked: a copy
    rm.ops.qk_norm_rope(qkv, 256, q, 128, None, 0, 9, 2, 1, 64, None, None, 0.0, None, None)
    rm.ops.qk_norm_rope(qkv, 256, q, 128, None, 0, 0, 2, 1, 64, None, None, 0.0, None, None)
    torch.cuda.synchronize()


def test_steps_of_no_tokens():
    none = {d: torch.empty(0, dtype=d, device="cuda") for d in (torch.bfloat16, torch.int32, torch.int64)}
    x, i32 = none[torch.bfloat16], none[torch.int32]
    pool = torch.zeros(2, 4 * 16 * 64, dtype=torch.bfloat16, device="cuda")
    cache = rm.KvCache(pool[0], pool[1], n_pages=4, page_size=16, n_kv_heads=1, head_dim=64)
    rope = rm.Rope(dev(C.rope_freqs(64, 1e4), torch.float64), 64)
    rm.ops.qk_norm_rope(x, 4 * 64, x, 128, x, 64, 0, 2, 1, 64, None, None, 0.0, rope, i32, cache, none[torch.int64])
    rm.ops.attn_window(x, 128, x, 64, x, 64, dev([0, 0], torch.int32), 1, 0, 2, 1, 64, 0, 0, x, 128)
    got = run_slots(np.array([5, 0]), np.array([0, 0]), np.arange(3), np.zeros((2, 1)), 0, 16, used=0)
    torch.cuda.synchronize()
    assert got[0].tolist() == [0, 0, 0] and got[3].tolist() == [5, 0] and got[4:6] == (0, 0) and (pool == 0).all()


def test_qk_norm_rope_keeps_nan_and_saturates():
    T, d = 4, 64
    qkv = randn((T, 3 * d), 3)
    qkv[1, d + 3] = NAN
    qkv[2, 2 * d + 5] = float("inf")
    pages = torch.zeros(2, 1, 16 * d, dtype=torch.uint8, device="cuda")
    one = torch.full((1,), 1e-3, device="cuda")
    cache = rm.KvCache(pages[0], pages[1], n_pages=1, page_size=16, n_kv_heads=1, head_dim=d, dtype=rm.E4M3, k_scale=one, v_scale=one)
    q, k = torch.empty(T, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    rm.ops.qk_norm_rope(qkv, 3 * d, q, d, k, d, T, 1, 1, d, None, None, 0.0, None, None, cache, torch.arange(T, device="cuda"))
    torch.cuda.synchronize()
    kk, vv = e4m3_pages(pages[0]).reshape(16, d), e4m3_pages(pages[1]).reshape(16, d)
    assert np.isnan(kk[1, 3]) and np.isnan(kk).sum() == 1 and torch.isnan(k[1, 3])
    assert vv[2, 5] == 448 and not np.isnan(vv).any() and np.abs(kk[0]).max() == 448


# --- attention over packed sequences ------------------------------------------------------

def window_case(lens, hq, hkv, d, window, sinks, seed=0, pad=0, extra=0, scale=1.0, poison=False, stream=None):
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    T = int(off[-1])
    q, k, v = (randn((T + extra, h * d + pad), seed + i, scale) for i, h in enumerate((hq, hkv, hkv)))
    if extra:                                     # rows behind the last sequence hold anything
        for t in (q, k, v):
            t[T:] = NAN
    out = torch.full((T + extra, hq * d + pad), -77.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    rm.ops.attn_window(q, hq * d + pad, k, hkv * d + pad, v, hkv * d + pad, dev(off, torch.int32), len(lens), T + extra, hq, hkv,
                       d, window, sinks, out, hq * d + pad, stream=stream)
    torch.cuda.synchronize()
    assert (out[T:] == -77.0).all() and (out[:, hq * d:] == -77.0).all()
    x = [f64(t)[:T, :h * d].reshape(T, h, d) for t, h in ((q, hq), (k, hkv), (v, hkv))]
    ref, mag, top = C.attend_window(*x, off, window, sinks)
    got = f64(out)[:T, :hq * d].reshape(T, hq, d)
    err, bound = np.abs(got - ref), attention_bound(ref, mag, top)
    assert np.all(err <= bound), (float(np.nanmax(err / bound)), np.argwhere(~(err <= bound))[:5])
    return out


@pytest.mark.parametrize("lens", [[1], [2], [0, 1, 0], [127], [128], [129], [255, 1, 0, 256], [3, 40, 100, 2, 7, 64, 65], [300, 513], [33] * 9])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (32, 4), (100, 1), (128, 128), (513, 3), (7, 200)])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (4, 1, 128)])
def test_attn_window(lens, window, sinks, hq, hkv, d):
    if sum(lens) > 0:
        window_case(lens, hq, hkv, d, window, sinks, seed=sum(lens))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (5, 1), (12, 4), (16, 1), (7, 1), (40, 2), (128, 1), (100, 1), (10, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_attn_window_head_layouts(hq, hkv, d):
    window_case([70, 1, 31, 150], hq, hkv, d, 50, 3, seed=hq)


@pytest.mark.parametrize("d", [64, 128])
def test_attn_window_of_nothing_writes_nothing(d):
    window_case([0, 0], 4, 2, d, 40, 2, extra=300)


@pytest.mark.parametrize("d,pad,extra", [(64, 8, 0), (128, 64, 5), (64, 0, 200), (128, 8, 1)])
def test_attn_window_strides_and_rows_behind(d, pad, extra):
    window_case([5, 131, 90], 4, 2, d, 40, 2, pad=pad, extra=extra)
    window_case([300], 2, 2, d, 0, 0, pad=pad, extra=extra)


@pytest.mark.parametrize("lens,hq", [([17], 8), ([100], 32), ([37], 64), ([65], 4), ([3, 97, 1], 16), ([200], 128)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (130, 1)])
def test_attn_window_nan_rows_behind_a_tile_of_one_token(lens, hq, d, window, sinks):
    # the last tile's warps all hold the last token: every key they are given is seen, what the MMA reads behind it is not
    window_case(lens, hq, 1, d, window, sinks, extra=40)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spoil", [False, True])
def test_attn_window_scores_of_minus_infinity(d, spoil):
    # keys whose score is -inf weigh nothing beside finite ones; rows that see no others are NaN (0 / 0)
    T, first = 300, 150
    q, k, v = torch.ones(T, d, dtype=torch.bfloat16, device="cuda"), randn((T, d), 4), randn((T, d), 5)
    k[:first, 3] = -float("inf")
    if spoil:
        v[T - 1] = NAN                            # rows before the last are computed again from what they see
    out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    rm.ops.attn_window(q, d, k, d, v, d, dev([0, T], torch.int32), 1, T, 1, 1, d, 0, 0, out, d)
    torch.cuda.synchronize()
    got, last = f64(out).reshape(T, 1, d), T - spoil
    x = [f64(t).reshape(T, 1, d)[first:last] for t in (q, k, v)]
    ref, mag, top = C.attend_window(*x, [0, last - first], 0, 0)
    assert np.isnan(got[:first]).all() and np.isnan(got[last:]).all()
    assert np.all(np.abs(got[first:last] - ref) <= attention_bound(ref, mag, top))


def window_on_device(q, k, v, off, window, sinks):
    """attend_window of the oracle in fp64 on the device, a sequence and a head at a time (for batches of many work items)."""
    T, hq, d = q.shape
    out, mag = torch.zeros(T, hq, d, dtype=torch.float64, device="cuda"), torch.zeros(T, hq, d, dtype=torch.float64, device="cuda")
    top = torch.zeros(T, hq, dtype=torch.float64, device="cuda")
    for a, b in zip(off[:-1], off[1:]):
        if a == b:
            continue
        i, j = torch.arange(b - a, device="cuda")[:, None], torch.arange(b - a, device="cuda")[None]
        seen = (j <= i) & ((j > i - window) | (j < sinks)) if window > 0 else j <= i
        for h in range(hq):
            kk, vv, qq = (x[a:b, y].double() for x, y in ((k, h // (hq // k.shape[1])), (v, h // (hq // k.shape[1])), (q, h)))
            p = torch.softmax((qq @ kk.T / d ** 0.5).masked_fill(~seen, -float("inf")), -1)
            out[a:b, h], mag[a:b, h] = p @ vv, p @ vv.abs()
            top[a:b, h] = ((qq.abs() @ kk.abs().T) / d ** 0.5).masked_fill(~seen, 0).amax(-1)
    return out.cpu().numpy(), mag.cpu().numpy(), top.cpu().numpy()


@pytest.mark.parametrize("n,lo,hi,hq,hkv,d,window,sinks", [
    (60, 1, 200, 12, 12, 64, 0, 0), (40, 100, 300, 16, 16, 128, 60, 4), (3, 900, 2500, 8, 1, 128, 300, 2),
    (200, 0, 40, 10, 10, 128, 16, 1), (9, 100, 900, 15, 3, 64, 200, 70), (400, 1, 3, 6, 2, 128, 0, 0)])
def test_attn_window_of_many_items(n, lo, hi, hq, hkv, d, window, sinks):
    # more work items than SMs: blocks take one after the other, tiles keep their barriers' turns across items
    lens = np.random.RandomState(n).randint(lo, hi + 1, n)
    off = np.concatenate([[0], np.cumsum(lens)])
    T = int(off[-1])
    q, k, v = (randn((T, h, d), n + i) for i, h in enumerate((hq, hkv, hkv)))
    ref, mag, top = window_on_device(q, k, v, off, window, sinks)
    dev_off = dev(off, torch.int32)
    outs = []
    for _ in range(3):
        out = torch.full((T, hq * d), NAN, dtype=torch.bfloat16, device="cuda")
        rm.ops.attn_window(q, hq * d, k, hkv * d, v, hkv * d, dev_off, n, T, hq, hkv, d, window, sinks, out, hq * d)
        outs.append(out)
    torch.cuda.synchronize()
    err, bound = np.abs(f64(outs[0]).reshape(T, hq, d) - ref), attention_bound(ref, mag, top)
    assert np.all(err <= bound), (float(np.nanmax(err / bound)), np.argwhere(~(err <= bound))[:3])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("n,lo,hi,hq,hkv,d,window,sinks", [
    (700, 1, 16, 8, 8, 64, 0, 0), (90, 129, 192, 6, 6, 64, 0, 0), (60, 200, 500, 4, 4, 128, 64, 1), (50, 300, 400, 12, 3, 64, 100, 64),
    (500, 1, 64, 16, 2, 128, 0, 0), (30, 600, 800, 8, 8, 64, 16, 16)])
def test_attn_window_chunks_of_few_keys(n, lo, hi, hq, hkv, d, window, sinks):
    # chunks of at most 64 keys (short sequences, ends, sinks) leave half of the softmax without keys: its warps keep
    # the tile's turns all the same
    test_attn_window_of_many_items(n, lo, hi, hq, hkv, d, window, sinks)


def test_attn_window_captured_replayed_and_on_two_streams():
    # a captured call on buffers that change, and two calls at once on streams of their own
    lens, hq, hkv, d = [200, 1, 77, 300], 8, 4, 128
    off = np.concatenate([[0], np.cumsum(lens)])
    T = int(off[-1])
    dev_off = dev(off, torch.int32)
    sets = [tuple(randn((T, h * d), 7 * s + i) for i, h in enumerate((hq, hkv, hkv))) for s in range(2)]

    def call(x, out, stream=None):
        rm.ops.attn_window(x[0], hq * d, x[1], hkv * d, x[2], hkv * d, dev_off, len(lens), T, hq, hkv, d, 50, 3, out, hq * d, stream=stream)

    want = []
    for x in sets:
        out = torch.empty(T, hq * d, dtype=torch.bfloat16, device="cuda")
        call(x, out)
        want.append(out)
    torch.cuda.synchronize()
    x = tuple(t.clone() for t in sets[0])
    out = torch.full_like(want[0], NAN)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        call(x, out, s)
    for which in (1, 0, 1):
        for a, b in zip(x, sets[which]):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[which])
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [torch.full_like(out, NAN), torch.full_like(out, NAN)]
    torch.cuda.synchronize()
    for _ in range(5):
        for y, o, st in zip(sets, outs, streams):
            call(y, o, st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@pytest.mark.parametrize("scale", [4.0, 20.0, 1e-3])
def test_attn_window_peaked_and_flat_rows(scale):
    # the scores' spread goes with scale^2: the running maximum moves often, or never
    window_case([400], 4, 4, 64, 0, 0, scale=scale)
    window_case([400], 4, 2, 128, 200, 4, scale=scale)


def test_attn_window_scores_that_climb():
    # each later key beats all earlier ones by far: every key tile raises the maximum
    T, d = 700, 128
    q = torch.ones(T, d, dtype=torch.bfloat16, device="cuda")
    k = (torch.arange(T, device="cuda")[:, None] * torch.ones(d, device="cuda") * 0.1).to(torch.bfloat16)
    v = randn((T, d), 3)
    out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    rm.ops.attn_window(q, d, k, d, v, d, dev([0, T], torch.int32), 1, T, 1, 1, d, 0, 0, out, d)
    torch.cuda.synchronize()
    x = [f64(t).reshape(T, 1, d) for t in (q, k, v)]
    ref, mag, top = C.attend_window(*x, [0, T], 0, 0)
    assert np.all(np.abs(f64(out).reshape(T, 1, d) - ref) <= attention_bound(ref, mag, top))


def test_attn_window_rows_computed_again_keep_nobody_waiting_too_long():
    # every row but a chunk's first is computed again, by one warp: the tile's other roles wait, and no wait gives up
    T, hq, hkv, d = 3000, 8, 2, 128
    q = torch.ones(T, hq * d, dtype=torch.bfloat16, device="cuda")
    k = (torch.arange(T, device="cuda")[:, None] * torch.ones(hkv * d, device="cuda") * 0.1).to(torch.bfloat16)
    v = randn((T, hkv * d), 3)
    out = torch.empty_like(q)
    rm.ops.attn_window(q, hq * d, k, hkv * d, v, hkv * d, dev([0, T], torch.int32), 1, T, hq, hkv, d, 0, 0, out, hq * d)
    torch.cuda.synchronize()
    assert rm.op_timeouts() == 0
    x = [t.view(T, h, d) for t, h in ((q, hq), (k, hkv), (v, hkv))]
    ref, mag, top = window_on_device(*x, [0, T], 0, 0)
    assert np.all(np.abs(f64(out).reshape(T, hq, d) - ref) <= attention_bound(ref, mag, top))


def test_attention_of_large_values():
    # values near the documented bounds, the window's under scores that climb
    T, d = 700, 128
    q = torch.ones(T, d, dtype=torch.bfloat16, device="cuda")
    k = (torch.arange(T, device="cuda")[:, None] * torch.ones(d, device="cuda") * 0.02).to(torch.bfloat16)
    v = (randn((T, d), 3) * 2.0 ** 70).to(torch.bfloat16)
    out = torch.empty_like(v)
    rm.ops.attn_window(q, d, k, d, v, d, dev([0, T], torch.int32), 1, T, 1, 1, d, 0, 0, out, d)
    torch.cuda.synchronize()
    x = [f64(t).reshape(T, 1, d) for t in (q, k, v)]
    ref, mag, top = C.attend_window(*x, [0, T], 0, 0)
    assert np.all(np.abs(f64(out).reshape(T, 1, d) - ref) <= attention_bound(ref, mag, top))
    v = (v.float() * 2.0 ** 40).to(torch.bfloat16)
    cache, _, _, table = paged([k[:, None]], [v[:, None]], 16, 4)
    space = torch.empty(rm.ops.attn_decode_workspace(1, 1, cache), dtype=torch.uint8, device="cuda")
    rm.ops.attn_decode(q[:1] * 0.01, d, cache, dev(table, torch.int32), table.shape[1], dev([T], torch.int32), 1, 1, 0, 0, out, d, space)
    torch.cuda.synchronize()
    ref, mag, top = C.attend(f64(q[:1] * 0.01), f64(k)[:, None], f64(v)[:, None], np.arange(T))
    assert np.all(np.abs(f64(out[:1]) - ref) <= attention_bound(ref, mag, top))


@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("d", [64, 128])
def test_attn_window_unseen_values_stay_out(bad, where, d):
    # a bad row in the middle: rows before it and rows whose window has passed it are as without it
    lens, hq, hkv, w = [60, 400, 90], 4, 2, 100
    off = np.concatenate([[0], np.cumsum(lens)])
    T, at = int(off[-1]), 60 + 150
    q, k, v = (randn((T, h * d), 5 + i) for i, h in enumerate((hq, hkv, hkv)))
    outs = []
    for spoil in (False, True):
        if spoil:
            (k if where == "k" else v)[at] = bad
        out = torch.empty(T, hq * d, dtype=torch.bfloat16, device="cuda")
        rm.ops.attn_window(q, hq * d, k, hkv * d, v, hkv * d, dev(off, torch.int32), 3, T, hq, hkv, d, w, 0, out, hq * d)
        torch.cuda.synchronize()
        outs.append(f64(out))
    rows = np.arange(T)
    sees = (rows >= at) & (rows < at + w)
    x = [f64(t).reshape(T, h, d) for t, h in ((q, hq), (k, hkv), (v, hkv))]
    clean = [np.where(np.isfinite(a), a, 0) for a in x]
    ref, mag, top = C.attend_window(*clean, off, w, 0)
    for o in outs:
        err = np.abs(o.reshape(T, hq, d) - ref)
        assert np.all(err[~sees] <= attention_bound(ref, mag, top)[~sees])
    if where == "v" or np.isnan(bad):
        assert not np.isfinite(outs[1][sees]).any()
    assert np.isfinite(outs[0]).all()


def test_attn_window_repeats_bit_for_bit_and_on_any_stream():
    a = window_case([513, 40, 1, 700], 8, 2, 128, 300, 4, seed=8)
    s = torch.cuda.Stream()
    for _ in range(3):
        assert torch.equal(a, window_case([513, 40, 1, 700], 8, 2, 128, 300, 4, seed=8, stream=s))


# --- attention of one new token over the cache ----------------------------------------------

def paged(k, v, page, seed, kind="bf16", gap=0, spare=3, width_extra=1):
    """Pages (shuffled, the unused slots NaN) of k, v: lists of [len][hkv][d] arrays."""
    hkv, d = k[0].shape[1:]
    need = [-(-len(a) // page) for a in k]
    ids = np.random.RandomState(seed).permutation(sum(need) + spare)
    width = max(1, max(need)) + width_extra
    table = np.full((len(k), width), 10 ** 6, dtype=np.int32)       # behind the sequence: numbers of no page
    shape = (sum(need) + spare, hkv * page * d + gap)
    pools = [torch.full(shape, NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    e = 0
    for i, m in enumerate(need):
        table[i, :m] = ids[e:e + m]
        e += m
        for pool, rows in zip(pools, (k[i], v[i])):
            for b in range(m):
                part = rows[b * page:(b + 1) * page].transpose(0, 1)
                pool[int(table[i, b]), :hkv * page * d].view(hkv, page, d)[:, :part.shape[1]] = part
    scales = [None, None]
    if kind == "e4m3":
        scales = [0.02 + 0.03 * torch.rand(hkv, generator=torch.Generator().manual_seed(seed + j)).cuda() for j in (1, 2)]
        out = []
        for pool, sc in zip(pools, scales):
            body = pool[:, :hkv * page * d].view(-1, hkv, page * d).float() / sc[None, :, None]
            enc = body.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(shape[0], -1)
            full = torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda")
            full[:, :hkv * page * d] = enc
            out.append(full)
        pools = out
    cache = rm.KvCache(*pools, n_pages=shape[0], page_size=page, n_kv_heads=hkv, head_dim=d,
                       dtype=rm.E4M3 if kind == "e4m3" else rm.BF16, k_scale=scales[0], v_scale=scales[1], page_stride=shape[1])
    return cache, pools, scales, table


def as_held(pools, scales, table, lens, page, hkv, d):
    """The cache's contents, sequence by sequence, in fp64 (what the oracle attends to)."""
    found = []
    for pool, sc in zip(pools, scales):
        x = pool[:, :hkv * page * d]
        x = e4m3_pages(x) if sc is not None else f64(x)
        x = x.reshape(-1, hkv, page, d)
        if sc is not None:
            x = x * f64(sc)[None, :, None, None]
        found.append([np.concatenate([x[table[i, b]].transpose(1, 0, 2) for b in range(-(-L // page))] + [np.zeros((0, hkv, d))])[:L]
                      for i, L in enumerate(lens)])
    return found


def decode_case(lens, hq, hkv, d, page, window=0, sinks=0, kind="bf16", seed=0, pad=0, gap=0, scale=1.0, stream=None):
    k = [randn((L, hkv, d), seed + 10 + i, scale) for i, L in enumerate(lens)]
    v = [randn((L, hkv, d), seed + 900 + i, scale) for i, L in enumerate(lens)]
    cache, pools, scales, table = paged(k, v, page, seed, kind, gap)
    n = len(lens)
    q = randn((n, hq * d + pad), seed, scale)
    out = torch.full((n, hq * d + pad), -77.0, dtype=torch.bfloat16, device="cuda")
    size = rm.ops.attn_decode_workspace(n, hq, cache)
    space = torch.full((size + 64,), 0xEE, dtype=torch.uint8, device="cuda")
    tab, length = dev(table, torch.int32), dev(lens, torch.int32)
    torch.cuda.synchronize()
    rm.ops.attn_decode(q, hq * d + pad, cache, tab, table.shape[1], length, n, hq, window, sinks, out, hq * d + pad, space, size,
                       stream=stream)
    torch.cuda.synchronize()
    assert (out[:, hq * d:] == -77.0).all() and (space[size:] == 0xEE).all()
    held = as_held(pools, scales, table, lens, page, hkv, d)
    qs, got = f64(q)[:, :hq * d].reshape(n, hq, d), f64(out)[:, :hq * d].reshape(n, hq, d)
    for i, L in enumerate(lens):
        ref, mag, top = C.attend(qs[i], held[0][i], held[1][i], C.seen_keys(L - 1, window, sinks))
        err, bound = np.abs(got[i] - ref), attention_bound(ref, mag, top)
        assert np.all(err <= bound), (i, L, float(np.nanmax(err / bound)))
    return out


@pytest.mark.parametrize("lens", [[1], [0], [2, 0, 17], [15, 16, 17, 63, 64, 65], [500], [3000, 1, 250], [129] * 40, [9000]])
@pytest.mark.parametrize("page", [1, 16, 24, 100])
@pytest.mark.parametrize("hq,hkv,d,kind", [(2, 2, 64, "bf16"), (8, 2, 128, "bf16"), (5, 1, 128, "e4m3"), (4, 4, 64, "e4m3")])
def test_attn_decode(lens, page, hq, hkv, d, kind):
    if page == 1 and sum(lens) > 3000:
        lens = [700]
    decode_case(lens, hq, hkv, d, page, kind=kind, seed=len(lens) + page)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (7, 1), (16, 1), (17, 1), (40, 2), (128, 1), (33, 1), (24, 8), (12, 12)])
@pytest.mark.parametrize("d,kind", [(64, "bf16"), (128, "bf16"), (64, "e4m3"), (128, "e4m3")])
def test_attn_decode_head_layouts(hq, hkv, d, kind):
    decode_case([70, 1, 333], hq, hkv, d, 32, kind=kind, seed=hq)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 3), (5000, 7), (64, 1000), (33, 33)])
@pytest.mark.parametrize("kind,d", [("bf16", 128), ("e4m3", 64)])
@pytest.mark.parametrize("page", [16, 48])
def test_attn_decode_window_and_sinks(window, sinks, kind, d, page):
    decode_case([1, 5, 16, 99, 100, 101, 640, 1500, 0], 4, 2, d, page, window, sinks, kind, seed=window)


@pytest.mark.parametrize("hq,hkv,d,kind", [(4, 4, 128, "bf16"), (24, 2, 64, "e4m3"), (8, 1, 128, "e4m3")])
def test_attn_decode_of_many_short_sequences_beside_a_long_one(hq, hkv, d, kind):
    # stretches of many units, and units over many stretches
    lens = [int(x) for x in np.random.RandomState(hq).randint(0, 70, 400)]
    lens[123] = 20000
    decode_case(lens, hq, hkv, d, 16, kind=kind, seed=1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attn_decode_strides(kind):
    decode_case([40, 700, 3], 4, 2, 64, 16, kind=kind, pad=8, gap=64)
    decode_case([40, 700, 3], 4, 2, 128, 16, kind=kind, pad=72, gap=16)


@pytest.mark.parametrize("scale", [6.0, 1e-3])
def test_attn_decode_peaked_and_flat(scale):
    decode_case([2000, 37], 8, 2, 128, 64, scale=scale)


def test_attn_decode_repeats_bit_for_bit_and_on_any_stream():
    a = decode_case([5000, 1, 77, 0, 1234], 8, 2, 128, 16, seed=3)
    s = torch.cuda.Stream()
    for _ in range(3):
        assert torch.equal(a, decode_case([5000, 1, 77, 0, 1234], 8, 2, 128, 16, seed=3, stream=s))


def test_attn_decode_drops_bad_pages_and_cuts_long_lengths():
    # page numbers of no page drop their tokens; a length beyond the row's pages is cut; a negative one sees nothing
    hq, hkv, d, page = 4, 2, 64, 16
    k, v = [randn((64, hkv, d), 1)] * 3, [randn((64, hkv, d), 2)] * 3
    cache, pools, scales, table = paged(k, v, page, 4, width_extra=0)
    table[0, 1], table[0, 2] = -5, 10 ** 9
    lens = [64, 10 ** 9, -3]
    q = randn((3, hq * d), 3)
    out = torch.full((3, hq * d), NAN, dtype=torch.bfloat16, device="cuda")
    space = torch.empty(rm.ops.attn_decode_workspace(3, hq, cache), dtype=torch.uint8, device="cuda")
    rm.ops.attn_decode(q, hq * d, cache, dev(table, torch.int32), 4, dev(lens, torch.int32), 3, hq, 0, 0, out, hq * d, space)
    torch.cuda.synchronize()
    qs, got = f64(q).reshape(3, hq, d), f64(out).reshape(3, hq, d)
    for i, seen in enumerate((np.r_[0:16, 48:64], np.arange(64), np.arange(0))):
        ref, mag, top = C.attend(qs[i], f64(k[0]), f64(v[0]), seen)
        assert np.all(np.abs(got[i] - ref) <= attention_bound(ref, mag, top))


def test_attn_decode_nothing_but_bad_pages_gives_zeros():
    cache, _, _, table = paged([randn((20, 1, 64), 1)], [randn((20, 1, 64), 2)], 16, 4)
    table[:] = -1
    out = torch.full((1, 64), NAN, dtype=torch.bfloat16, device="cuda")
    space = torch.empty(rm.ops.attn_decode_workspace(1, 1, cache), dtype=torch.uint8, device="cuda")
    rm.ops.attn_decode(randn((1, 64), 3), 64, cache, dev(table, torch.int32), table.shape[1], dev([20], torch.int32), 1, 1, 0, 0, out,
                       64, space)
    torch.cuda.synchronize()
    assert (out == 0).all()


def test_attn_decode_window_reads_no_hidden_page():
    # pages wholly outside the window and the sinks may be anything, numbers of no page among them
    hq, hkv, d, page, L = 2, 1, 64, 16, 400
    k, v = randn((L, hkv, d), 1), randn((L, hkv, d), 2)
    cache, pools, scales, table = paged([k], [v], page, 4)
    table[0, 1:(L - 50) // page] = -1
    q = randn((1, hq * d), 3)
    out = torch.empty(1, hq * d, dtype=torch.bfloat16, device="cuda")
    space = torch.empty(rm.ops.attn_decode_workspace(1, hq, cache), dtype=torch.uint8, device="cuda")
    rm.ops.attn_decode(q, hq * d, cache, dev(table, torch.int32), table.shape[1], dev([L], torch.int32), 1, hq, 50, 5, out, hq * d, space)
    torch.cuda.synchronize()
    ref, mag, top = C.attend(f64(q).reshape(hq, d), f64(k), f64(v), C.seen_keys(L - 1, 50, 5))
    assert np.all(np.abs(f64(out).reshape(hq, d) - ref) <= attention_bound(ref, mag, top))


def test_attn_decode_infinite_scores_in_a_seen_key_are_nan_as_defined():
    # a NaN that IS seen reaches its row, and no other row
    cache, pools, _, table = paged([randn((40, 1, 64), 1), randn((40, 1, 64), 5)], [randn((40, 1, 64), 2), randn((40, 1, 64), 6)], 16, 4)
    pools[1][int(table[1, 0]), 3] = NAN
    out = torch.empty(2, 64, dtype=torch.bfloat16, device="cuda")
    space = torch.empty(rm.ops.attn_decode_workspace(2, 1, cache), dtype=torch.uint8, device="cuda")
    rm.ops.attn_decode(randn((2, 64), 3), 64, cache, dev(table, torch.int32), table.shape[1], dev([40, 40], torch.int32), 2, 1, 0, 0, out,
                       64, space)
    torch.cuda.synchronize()
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1, 3]) and torch.isfinite(out[1, :3]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L,first", [(1, 1), (40, 40), (300, 299), (300, 150), (5000, 5000), (5000, 4990)])
def test_attn_decode_scores_of_minus_infinity(d, L, first):
    # as in the windowed attention: -inf weighs nothing beside a finite score, and nothing else to see is NaN
    k, v = randn((L, 1, d), 4), randn((L, 1, d), 5)
    k[:first, 0, 3] = -float("inf")
    cache, _, _, table = paged([k], [v], 16, 4)
    q = torch.ones(1, d, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(1, d, dtype=torch.bfloat16, device="cuda")
    space = torch.empty(rm.ops.attn_decode_workspace(1, 1, cache), dtype=torch.uint8, device="cuda")
    rm.ops.attn_decode(q, d, cache, dev(table, torch.int32), table.shape[1], dev([L], torch.int32), 1, 1, 0, 0, out, d, space)
    torch.cuda.synchronize()
    if first == L:
        assert torch.isnan(out).all()
    else:
        ref, mag, top = C.attend(f64(q), f64(k)[first:], f64(v)[first:], np.arange(L - first))
        assert np.all(np.abs(f64(out) - ref) <= attention_bound(ref, mag, top))


@pytest.mark.parametrize("below", [18, 26, 30])
@pytest.mark.parametrize("n,L,hq", [(1, 32, 1), (600, 1000, 1), (300, 500, 12)])
@pytest.mark.parametrize("d", [64, 128])
def test_attn_decode_8_bit_cache_of_a_dominant_key_and_a_flat_tail(d, n, L, hq, below):
    # one key's weight is 2^below times each other's, and its value is 0: the output is the tail's share alone
    k, v = torch.zeros(L, d, device="cuda"), randn((L, d), 5).float()
    k[:, 0], k[0, 0], v[0] = -2.0, 16.0, 0.0
    pages = -(-L // 16)
    pools = [torch.full((pages * 16, d), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for pool, x in zip(pools, (k, v)):
        pool[:L] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    cache = rm.KvCache(*pools, n_pages=pages, page_size=16, n_kv_heads=1, head_dim=d, dtype=rm.E4M3)
    q = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = below * np.log(2) * d ** 0.5 / 18
    out = torch.empty(n, hq * d, dtype=torch.bfloat16, device="cuda")
    space = torch.empty(rm.ops.attn_decode_workspace(n, hq, cache), dtype=torch.uint8, device="cuda")
    table = dev(np.tile(np.arange(pages), (n, 1)), torch.int32)
    rm.ops.attn_decode(q, hq * d, cache, table, pages, dev([L] * n, torch.int32), n, hq, 0, 0, out, hq * d, space)
    torch.cuda.synchronize()
    held = [e4m3_pages(pool)[:L, None] for pool in pools]
    ref, mag, top = C.attend(f64(q[0]), *held, np.arange(L))
    err, bound = np.abs(f64(out).reshape(n, hq, d) - ref), attention_bound(ref, mag, top)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (0, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)])
def test_attention_of_the_largest_windows_and_sinks(window, sinks):
    window_case([1, 300, 129], 4, 2, 64, window, sinks)
    decode_case([1, 300, 129, 0], 4, 2, 64, 16, window, sinks)


def test_offsets_beyond_32_bits():
    # a cache of over 2^32 elements: pages at its two ends, written through slots and read back
    hkv, d, page = 8, 128, 16
    per = hkv * d * page
    n_pages = (2 ** 32 + 2 ** 20) // per
    k, v = (torch.empty(n_pages, per, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = rm.KvCache(k, v, n_pages=n_pages, page_size=page, n_kv_heads=hkv, head_dim=d)
    L = 40
    pages = [n_pages - 1, 0, n_pages - 2]
    qkv = randn((L, 24 * d), 1)
    slots = np.array([pages[t // page] * page + t % page for t in range(L)])
    q = torch.empty(L, hkv * d, dtype=torch.bfloat16, device="cuda")
    rm.ops.qk_norm_rope(qkv, 24 * d, q, hkv * d, None, 0, L, hkv, hkv, d, None, None, 0.0, None, None, cache, dev(slots, torch.int64))
    out = torch.empty(1, hkv * d, dtype=torch.bfloat16, device="cuda")
    space = torch.empty(rm.ops.attn_decode_workspace(1, hkv, cache), dtype=torch.uint8, device="cuda")
    rm.ops.attn_decode(q[L - 1:], hkv * d, cache, dev([pages], torch.int32), 3, dev([L], torch.int32), 1, hkv, 0, 0, out, hkv * d, space)
    torch.cuda.synchronize()
    x = f64(qkv).reshape(L, 3, hkv, d)
    ref, mag, top = C.attend(x[L - 1, 0], x[:, 1], x[:, 2], np.arange(L))
    assert np.all(np.abs(f64(out).reshape(hkv, d) - ref) <= attention_bound(ref, mag, top))


# --- waits that give up ---------------------------------------------------------------------

def test_a_wait_that_gives_up_is_counted_and_told_once():
    # no kernel of the tests before gave one up; one that nothing ends is told, and the operators go on working
    assert rm.op_timeouts() == 0
    rm.selftest_op_wait(2_000_000)
    rm.selftest_op_wait(2_000_000)
    assert rm.op_timeouts() == 2
    window_case([300, 20], 4, 2, 128, 100, 4)
    assert rm.op_timeouts() == 0


@pytest.fixture(scope="module", autouse=True)
def no_wait_gives_up(cuda):
    yield
    assert rm.op_timeouts() == 0 and rm.bounds_errors() == 0      # (the second counts in the checked build alone)


# --- what the device check refuses ---------------------------------------------------------

def test_host_pointers_are_refused():
    host = torch.zeros(1 << 16, dtype=torch.bfloat16)
    onda = torch.zeros(1 << 16, dtype=torch.bfloat16, device="cuda")
    off = dev([0, 5], torch.int32)
    good = dict(q=onda, q_stride=64, k=onda, k_stride=64, v=onda, v_stride=64, offsets_dev=off, n_seqs=1, T=5, n_q_heads=1,
                n_kv_heads=1, head_dim=64, window=0, sinks=0, out=onda.clone(), out_stride=64)
    rm.ops.attn_window(**good)
    for name in ("q", "k", "v", "out", "offsets_dev"):
        with pytest.raises(rm.RmError) as e:
            rm.ops.attn_window(**{**good, name: host})
        assert e.value.code == rm.RM_E_INVAL
    torch.cuda.synchronize()


# --- a run of them together ---------------------------------------------------------------

def project(x, w):
    """The QKV projection of the step (rm_op_gemm)."""
    y = torch.empty(x.shape[0], w.shape[0], dtype=torch.bfloat16, device="cuda")
    rm.ops.gemm(x, w, None, y, rm.BF16, x.shape[0], w.shape[0], w.shape[1])
    return y


class Stepper:
    """One attention layer of a growing batch: every buffer of its steps, as a program would hold them."""

    def __init__(self, n, hq, hkv, d, page, n_pages, width, window, sinks, kind, hidden, seed):
        self.n, self.hq, self.hkv, self.d, self.page, self.window, self.sinks = n, hq, hkv, d, page, window, sinks
        self.w = randn(((hq + 2 * hkv) * d, hidden), seed, hidden ** -0.5)
        self.q_gain, self.k_gain = (1 + 0.1 * torch.randn(d, generator=torch.Generator().manual_seed(seed + i)).cuda() for i in (1, 2))
        self.freqs = rm.ops.rope_freqs(d // 2, 1000.0, rm.ROPE_PARTS, 4.0, 256, 32, 1)
        self.rope = rm.Rope(dev(self.freqs, torch.float64), d // 2, layout=rm.ROPE_HALF)
        f8 = kind == "e4m3"
        self.pools = [torch.full((n_pages, hkv * page * d), 0x7f if f8 else NAN, dtype=torch.uint8 if f8 else torch.bfloat16,
                                 device="cuda") for _ in range(2)]
        self.scales = [torch.full((hkv,), 0.03, device="cuda") for _ in range(2)] if f8 else [None, None]
        self.cache = rm.KvCache(*self.pools, n_pages=n_pages, page_size=page, n_kv_heads=hkv, head_dim=d,
                                dtype=rm.E4M3 if f8 else rm.BF16, k_scale=self.scales[0], v_scale=self.scales[1])
        i32 = dict(dtype=torch.int32, device="cuda")
        self.length, self.used = torch.zeros(n, **i32), torch.zeros(1, **i32)
        self.table = torch.full((n, width), -1, **i32)
        self.free = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
        self.offsets, self.unserved = torch.zeros(n + 1, **i32), torch.zeros(1, **i32)
        self.space = torch.empty(rm.ops.attn_decode_workspace(n, hq, self.cache), dtype=torch.uint8, device="cuda")
        self.one = torch.ones(n, **i32)

    def buffers(self, T):
        b = dict(dtype=torch.bfloat16, device="cuda")
        return {"positions": torch.empty(T, dtype=torch.int32, device="cuda"), "slots": torch.empty(T, dtype=torch.int64, device="cuda"),
                "q": torch.empty(T, self.hq * self.d, **b), "k": torch.empty(T, self.hkv * self.d, **b),
                "out": torch.full((T, self.hq * self.d), NAN, **b)}

    def prepare(self, x, new, b, stream=None):
        T, hall = x.shape[0], self.hq + 2 * self.hkv
        rm.ops.kv_slots(self.length, new, self.n, self.page, self.free, self.free.numel(), self.used, self.table, self.table.shape[1],
                        T, self.offsets, b["positions"], b["slots"], self.length, self.used, self.unserved, stream=stream)
        y = torch.empty(T, hall * self.d, dtype=torch.bfloat16, device="cuda") if "qkv" not in b else b["qkv"]
        rm.ops.gemm(x, self.w, None, y, rm.BF16, T, hall * self.d, self.w.shape[1], stream=stream)
        rm.ops.qk_norm_rope(y, hall * self.d, b["q"], self.hq * self.d, b["k"], self.hkv * self.d, T, self.hq, self.hkv, self.d,
                            self.q_gain, self.k_gain, 1e-6, self.rope, b["positions"], self.cache, b["slots"], stream=stream)
        return y

    def prompt(self, x, new):
        b = self.buffers(x.shape[0])
        y = self.prepare(x, new, b)
        v = y[:, (self.hq + self.hkv) * self.d:]
        rm.ops.attn_window(b["q"], self.hq * self.d, b["k"], self.hkv * self.d, v, y.shape[1], self.offsets, self.n, x.shape[0], self.hq,
                           self.hkv, self.d, self.window, self.sinks, b["out"], self.hq * self.d)
        return b

    def step(self, x, b, stream=None):
        self.prepare(x, self.one, b, stream)
        rm.ops.attn_decode(b["q"], self.hq * self.d, self.cache, self.table, self.table.shape[1], self.length, self.n, self.hq,
                           self.window, self.sinks, b["out"], self.hq * self.d, self.space, stream=stream)


@pytest.mark.parametrize("window,sinks,kind", [(0, 0, "bf16"), (40, 3, "bf16"), (0, 0, "e4m3"), (64, 4, "e4m3")])
@pytest.mark.parametrize("graph", [False, True])
def test_prompts_then_steps_like_the_whole_texts(window, sinks, kind, graph):
    """Prompts, then steps one token at a time (eagerly, or one captured step
    replayed), against each text attended to as a whole in fp64 from its
    projections: the cache, the slot maps and both attentions agree."""
    n, hq, hkv, d, page, hidden, steps = 5, 8, 2, 64, 16, 64, 20
    lens = [1, 77, 16, 130, 33]
    S = Stepper(n, hq, hkv, d, page, 60, 16, window, sinks, kind, hidden, 11)
    T = sum(lens)
    x0 = randn((T, hidden), 21)
    xs = [randn((n, hidden), 30 + i) for i in range(steps)]
    b0 = S.prompt(x0, dev(lens, torch.int32))
    qs = [[b0["q"]], []]
    outs = []
    b = S.buffers(n)
    b["qkv"] = torch.empty(n, (hq + 2 * hkv) * d, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(n, hidden, dtype=torch.bfloat16, device="cuda")
    if graph:
        state = [t.clone() for t in (S.length, S.used, S.table, *S.pools)]
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        x.copy_(xs[0])
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            S.step(x, b, stream=s)
        torch.cuda.synchronize()
        for t, was in zip((S.length, S.used, S.table, *S.pools), state):
            assert torch.equal(t.view(torch.uint8), was.view(torch.uint8))         # capturing ran nothing
    for i in range(steps):
        x.copy_(xs[i])
        if graph:
            g.replay()
        else:
            S.step(x, b)
        outs.append((b["q"].clone(), b["k"].clone(), b["qkv"].clone(), b["out"].clone()))
    torch.cuda.synchronize()
    assert int(S.unserved) == 0 and S.length.tolist() == [L + steps for L in lens]
    assert int(S.used) == sum(-(-(L + steps) // page) for L in lens)
    held = as_held(S.pools, S.scales, S.table.cpu().numpy(), [L + steps for L in lens], page, hkv, d)
    off = np.concatenate([[0], np.cumsum(lens)])
    # the cache holds the tokens' keys (as k_out gave them) and values, in order
    for i, L in enumerate(lens):
        keys = np.concatenate([f64(b0["k"])[off[i]:off[i + 1]]] + [f64(o[1])[i:i + 1] for o in outs]).reshape(-1, hkv, d)
        if kind == "bf16":
            assert np.array_equal(held[0][i], keys)
        else:
            assert np.all(np.abs(held[0][i] - keys) <= (HALF_E4M3 + 2 * HALF_BF16) * np.abs(keys) + 0.03 * 2.0 ** -10 + 1e-5)
    # positions and rotation: the rotated keys are the projections' at their positions
    pos = np.concatenate([np.arange(L) for L in lens])
    y = f64(project(x0, S.w)).reshape(T, -1, d)
    rk, mk = C.norm_rope(y[:, hq:hq + hkv], f64(S.k_gain), 1e-6, pos, S.freqs, 0)
    assert np.all(np.abs(f64(b0["k"]).reshape(T, hkv, d) - rk) <= HALF_BF16 * np.abs(rk) + 2 * F32_RTOL * mk)
    # prompts
    q0, v0 = f64(b0["q"]).reshape(T, hq, d), y[:, hq + hkv:]
    ref, mag, top = C.attend_window(q0, f64(b0["k"]).reshape(T, hkv, d), v0, off, window, sinks)
    assert np.all(np.abs(f64(b0["out"]).reshape(T, hq, d) - ref) <= attention_bound(ref, mag, top))
    # steps, each over the cache as it stood
    for j, (q, _, _, o) in enumerate(outs):
        for i, L in enumerate(lens):
            seen = C.seen_keys(L + j, window, sinks)
            ref, mag, top = C.attend(f64(q[i]).reshape(hq, d), held[0][i], held[1][i], seen)
            assert np.all(np.abs(f64(o[i]).reshape(hq, d) - ref) <= attention_bound(ref, mag, top)), (j, i)


@pytest.mark.parametrize("graph", [False, True])
def test_two_batches_at_once_on_streams_of_their_own(graph):
    """Prompts and steps of two batches interleaved on two streams (eagerly, or
    as two captured steps replayed at once) give what each gives alone."""
    n, hidden, steps = 70, 64, 12
    lens = np.random.RandomState(3).randint(1, 200, n)
    kinds = (("bf16", 0, 0), ("e4m3", 50, 3))

    def batch(which):
        kind, window, sinks = kinds[which]
        return Stepper(n, 8, 2, 128, 16, 1200, 16, window, sinks, kind, hidden, 40 + which)

    xs = [[randn((int(lens.sum()), hidden), 50 + w)] + [randn((n, hidden), 60 + 20 * w + i) for i in range(steps)] for w in range(2)]
    new = dev(lens, torch.int32)

    def go(S, w, streams):
        b, x = S.buffers(n), torch.empty(n, hidden, dtype=torch.bfloat16, device="cuda")
        b["qkv"] = torch.empty(n, 12 * 128, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph() if graph else None
        if graph:
            x.copy_(xs[w][1])
            torch.cuda.synchronize()
            with torch.cuda.graph(g, stream=streams[w]):
                S.step(x, b, stream=streams[w])
        with torch.cuda.stream(streams[w]):
            p = S.buffers(xs[w][0].shape[0])
            y = S.prepare(xs[w][0], new, p, stream=streams[w])
            rm.ops.attn_window(p["q"], 1024, p["k"], 256, y[:, 10 * 128:], y.shape[1], S.offsets, n, y.shape[0], 8, 2, 128, S.window,
                               S.sinks, p["out"], 1024, stream=streams[w])
            outs = [p["out"]]
        for i in range(steps):
            with torch.cuda.stream(streams[w]):
                x.copy_(xs[w][1 + i])
                if graph:
                    g.replay()
                else:
                    S.step(x, b, stream=streams[w])
                outs.append(b["out"].clone())
            yield None
        yield outs + [S.length, S.used, S.table, *S.pools, y, x, g]

    alone = []
    for w in range(2):
        alone.append([o for o in go(batch(w), w, [torch.cuda.Stream(), torch.cuda.Stream()])][-1])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    runs = [go(batch(w), w, streams) for w in range(2)]
    both = [None, None]
    for _ in range(steps + 1):
        both = [next(r) for r in runs]
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a[:-1], b[:-1]))


def test_a_prompt_scored_whole_and_token_by_token_agree():
    """The window attention over a text and the decode attention of each of
    its tokens in turn round alike up to their tolerances."""
    L, hq, hkv, d, page = 90, 4, 2, 128, 16
    q, k, v = randn((L, hq * d), 1), randn((L, hkv * d), 2), randn((L, hkv * d), 3)
    whole = torch.empty_like(q)
    rm.ops.attn_window(q, hq * d, k, hkv * d, v, hkv * d, dev([0, L], torch.int32), 1, L, hq, hkv, d, 25, 2, whole, hq * d)
    cache, pools, _, table = paged([k.view(L, hkv, d)], [v.view(L, hkv, d)], page, 5, width_extra=0)
    tab = dev(np.repeat(table, L, axis=0), torch.int32)                 # one row per prefix of the text
    each = torch.empty_like(q)
    space = torch.empty(rm.ops.attn_decode_workspace(L, hq, cache), dtype=torch.uint8, device="cuda")
    rm.ops.attn_decode(q, hq * d, cache, tab, table.shape[1], dev(np.arange(1, L + 1), torch.int32), L, hq, 25, 2, each, hq * d, space)
    torch.cuda.synchronize()
    x = [f64(t).reshape(L, h, d) for t, h in ((q, hq), (k, hkv), (v, hkv))]
    ref, mag, top = C.attend_window(*x, [0, L], 25, 2)
    assert np.all(np.abs(f64(whole) - f64(each)).reshape(L, hq, d) <= 2 * attention_bound(ref, mag, top))
