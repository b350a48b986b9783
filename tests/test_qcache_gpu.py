"""GPU: the 8-bit latent cache against its definition in 64 bits.

Tolerances, derived:
  * scales are powers of two (or the caller's) and have to be equal;
  * a stored value is one rounding to e4m3 (half a step: 2^-4 of the value, or half of the
    smallest step 2^-9 below the normals) of the row's value, which the kernel holds to a
    few fp32 roundings (2^-22 here): |stored - x / s| <= 2^-4 |x / s| (1 + 2^-18) or 2^-10;
  * values read back: one fp32 product (2^-24) and one rounding to the output's type;
  * expanded heads: 512 fp32 additions of exact products (512 * 2^-24 of the sum of
    magnitudes; the fp32 path's products round as well: twice that) and the output's rounding;
  * decode: the framework's parity bar over the values that the cache holds.
"""
import numpy as np
import pytest
import torch

import differential_latent_attention_gdla_b200 as gdla
import oracle
from differential_latent_attention_gdla_b200 import _abi
from differential_latent_attention_gdla_b200 import workloads as wl
from gdla_testutil import assert_parity, f64, mask_code, oracle_prefill_rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def gen_for(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def scale_of(amax):
    """The smallest power of two, at least 2^-40, with amax <= 448 s."""
    e = -40
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def e4m3_values(t):
    return t.view(torch.float8_e4m3fn).cpu().double().numpy()


def token_scales(scales, nb, T):
    return np.repeat(f64(scales), nb, axis=1)[:, :T]


def held(c8, kr8, scales, nb):
    """The values that a cache holds, in 64 bits: [B, T, d_c + d_rope]."""
    v = np.concatenate([e4m3_values(c8), e4m3_values(kr8)], -1)
    return v * token_scales(scales, nb, c8.shape[1])[..., None]


def new_rows(c_kv, k_rope, gamma, cos, sin, start, eps=1e-6):
    """The rows before quantisation, in 64 bits: [B, L, d_c + d_rope]."""
    c, k = f64(c_kv), f64(k_rope)
    if gamma is None:
        return np.concatenate([c, k], -1)
    c = c / np.sqrt((c * c).mean(-1, keepdims=True) + eps) * f64(gamma)
    half = k.shape[-1] // 2
    out = np.zeros_like(k)
    for b in range(k.shape[0]):
        for i in range(k.shape[1]):
            p = min(start[b] + i, cos.shape[0] - 1)
            cs, sn = f64(cos[p]), f64(sin[p])
            out[b, i, :half] = k[b, i, :half] * cs - k[b, i, half:] * sn
            out[b, i, half:] = k[b, i, half:] * cs + k[b, i, :half] * sn
    return np.concatenate([c, out], -1)


def assert_quantised(stored, x, s):
    """stored (e4m3 values) is x / s, rounded."""
    y = np.abs(x / s)
    bound = np.maximum(2.0 ** -4 * y * (1 + 2.0 ** -18), 2.0 ** -10 * (1 + 2.0 ** -18))
    assert np.isfinite(stored).all()
    err = np.abs(stored - x / s)
    assert (err <= bound).all(), float((err - bound).max())


# ------------------------------------------------------------------------ write
WRITES = [
    # d_c, d_rope, dtype, T, L, scale_block, start, lens
    (512, 64, "bf16", 300, 1, 1, [0, 299, 17], [1, 1, 1]),          # a step
    (512, 64, "bf16", 300, 1, 64, [0, 299, 64], [1, 1, 0]),         # a step inside blocks; an empty slot
    (512, 64, "bf16", 257, 200, 16, [0, 57, 13], [200, 200, 187]),  # chunks that begin and end inside blocks
    (512, 64, "fp32", 257, 200, 16, [3, 57, 31], [199, 1, 0]),
    (512, 64, "bf16", 260, 260, 128, [0, 100, 129], [260, 160, 131]),
    (512, 64, "fp32", 260, 260, 128, [0, 127, 128], [260, 133, 132]),
    (512, 64, "bf16", 100, 100, 32, [0, 0, 99], [100, 33, 1]),
    (512, 64, "fp32", 130, 65, 64, [0, 1, 65], [65, 64, 63]),
    (256, 32, "bf16", 77, 50, 2, [0, 27, 1], [50, 50, 49]),
    (256, 32, "fp32", 77, 50, 4, [0, 27, 3], [50, 50, 0]),
    (128, 64, "bf16", 65, 65, 8, [0, 5, 64], [65, 60, 1]),
    (64, 16, "bf16", 33, 33, 1, [0, 32, 33], [33, 1, 0]),
    (64, 16, "fp32", 1, 1, 1, [0, 0, 0], [1, 1, 0]),
    (64, 16, "fp32", 1, 1, 128, [0, 0, 1], [1, 0, 0]),
]


# the kernel of many bf16 tokens (16384 and more): chunks of whole blocks, ragged at both ends
MANY = [
    (512, 64, "bf16", 7000, 6000, 1, [0, 999, 1000], [6000, 5990, 0]),
    (512, 64, "bf16", 7000, 6000, 16, [5, 1000, 37], [5999, 6000, 5000]),
    (512, 64, "bf16", 7000, 6000, 64, [63, 64, 65], [6000, 1, 5937]),
    (256, 32, "bf16", 7000, 6000, 2, [1, 0, 77], [6000, 6000, 3]),
    (64, 16, "bf16", 7000, 6000, 32, [0, 31, 1000], [5985, 6000, 6000]),
]


@pytest.mark.parametrize("d_c,d_rope,dt,T,L,nb,start,lens", WRITES + MANY)
@pytest.mark.parametrize("norm", [True, False])
def test_write(d_c, d_rope, dt, T, L, nb, start, lens, norm):
    B, gen, dtype = 3, gen_for(T * 131 + L), DT[dt]
    n_blocks = gdla.qcache_scale_blocks(T, nb)
    c_kv = (torch.randn((B, L, d_c), generator=gen) * torch.exp2(torch.randint(-12, 12, (B, L, 1), generator=gen))).to(dtype)
    k_rope = torch.randn((B, L, d_rope), generator=gen).to(dtype)
    gamma = (1 + 0.2 * torch.randn(d_c, generator=gen)).to(dtype) if norm else None
    cos, sin = gdla.rope_tables(T, d_rope, device=DEV)
    # earlier tokens: any bytes that are numbers, and scales of the same range
    c8 = torch.randint(0, 120, (B, T, d_c), generator=gen, dtype=torch.uint8).to(DEV)
    kr8 = torch.randint(128, 248, (B, T, d_rope), generator=gen, dtype=torch.uint8).to(DEV)
    scales = torch.exp2(torch.randint(-12, 2, (B, n_blocks), generator=gen).float()).to(DEV)
    was, was_s = [c8.clone(), kr8.clone()], f64(scales)
    ws = torch.full((256,), 0x55, dtype=torch.uint8, device=DEV)
    gdla.qcache_write(c8, kr8, scales, c_kv.to(DEV), k_rope.to(DEV), gamma=gamma.to(DEV) if norm else None, rope_cos=cos,
                      rope_sin=sin, start=i32(start), lens=i32(lens), scale_block=nb, workspace=ws)
    assert gdla.workspace_status(ws) == _abi.GDLA_OK
    x = new_rows(c_kv, k_rope, gamma, cos, sin, start)
    got_s = f64(scales)
    old = np.concatenate([e4m3_values(t) for t in was], -1)
    new = np.concatenate([e4m3_values(c8), e4m3_values(kr8)], -1)
    for b in range(B):
        p0, p1 = start[b], start[b] + lens[b]
        touched = range(p0 // nb, (p1 + nb - 1) // nb) if lens[b] else ()
        for k in range(n_blocks):
            if k not in touched:
                assert got_s[b, k] == was_s[b, k]
                continue
            lo, hi = max(k * nb, p0), min((k + 1) * nb, p1)
            want = scale_of(np.abs(x[b, lo - p0:hi - p0]).max())
            if k * nb < p0:
                want = max(want, was_s[b, k])
                assert_quantised(new[b, k * nb:p0], old[b, k * nb:p0] * was_s[b, k], want)
            assert got_s[b, k] == want, (b, k)
            assert_quantised(new[b, lo:hi], x[b, lo - p0:hi - p0], want)
        # rows in front of the first touched block and behind the last new token: as they were
        first = p0 // nb * nb if lens[b] else T
        for now, before in zip((c8, kr8), was):
            assert torch.equal(now[b, :first], before[b, :first])
            assert torch.equal(now[b, p1 if lens[b] else T:], before[b, p1 if lens[b] else T:])


def test_write_scale_borders_and_extremes():
    # one token a block, rows already normalised: maxima at and next to 448 2^e, zeros, the
    # smallest and largest values
    top = [448.0, 448.0001, 447.9999, 448 * 2.0 ** -9, np.nextafter(np.float32(448 * 2.0 ** -9), np.float32(1)), 0.0,
           1e-30, 2.0 ** -40 * 448, 2.0 ** -41 * 448, 1e-45, 3e38, 1.0]
    n = len(top)
    c = torch.zeros((1, n, 64))
    for i, v in enumerate(top):
        c[0, i, i] = float(-v if i % 2 else v)
    k = torch.zeros((1, n, 16))
    c8, kr8, sc = gdla.qcache_empty(1, n, d_c=64, d_rope=16, device=DEV)
    gdla.qcache_write(c8, kr8, sc, c.to(DEV), k.to(DEV))
    want = np.array([scale_of(abs(float(c[0, i].abs().max()))) for i in range(n)])
    assert (f64(sc)[0] == want).all()
    assert_quantised(e4m3_values(c8)[0], f64(c)[0], want[:, None])
    assert (kr8.view(torch.uint8).cpu() == 0).all()
    # the same over the rotary part
    c8, kr8, sc = gdla.qcache_empty(1, n, d_c=64, d_rope=16, device=DEV)
    k[0, :, 3] = torch.tensor([float(c[0, i].abs().max()) for i in range(n)])
    gdla.qcache_write(c8, kr8, sc, torch.zeros((1, n, 64), device=DEV), k.to(DEV))
    assert (f64(sc)[0] == want).all()


@pytest.mark.parametrize("dt,B,L", [("bf16", 1, 64), ("fp32", 1, 64), ("bf16", 3, 6000)])
def test_write_scales_next_to_their_borders(dt, B, L):
    # normalised maxima within 1e-6 of 448 2^e = 0.875 on either side: rows of equal magnitudes a
    # give gamma / sqrt(1 + eps / a^2), and a last element a little larger or smaller moves it
    gen = gen_for(60)
    a = torch.exp2(torch.randint(-3, 12, (B, L, 1), generator=gen).float())
    c = a * (torch.randint(0, 2, (B, L, 64), generator=gen) * 2 - 1)
    if dt == "fp32":
        c[..., -1] *= 1 + 2.0 ** -20 * torch.randint(-8, 9, (B, L), generator=gen)
    else:  # (one larger element among the small ones; the gain makes up for it)
        c[..., -1] *= 1 + 2.0 ** -7 * torch.randint(0, 2, (B, L), generator=gen)
    c = c.to(DT[dt])
    gamma = torch.full((64,), 0.875).to(DT[dt])
    gamma[-1] = 0.5
    k = torch.zeros((B, L, 16), dtype=DT[dt])
    cos, sin = gdla.rope_tables(L, 16, device=DEV)
    cache = gdla.qcache_empty(B, L, d_c=64, d_rope=16, device=DEV)
    gdla.qcache_write(*cache, c.to(DEV), k.to(DEV), gamma=gamma.to(DEV), rope_cos=cos, rope_sin=sin)
    x = f64(c)
    x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * f64(gamma)
    top = np.abs(x).max(-1)
    want = np.where(top <= 0.875, 2.0 ** -9, 2.0 ** -8)
    assert (np.abs(top - 0.875) < 1e-3).all() and (want == 2.0 ** -9).any()
    assert (f64(cache[2]) == want).all()
    assert_quantised(e4m3_values(cache[0]), x, want[..., None])


@pytest.mark.parametrize("T", [40, 16400])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_write_not_finite_values_stay_apart(dt, T):
    # a NaN or infinity is stored as NaN; the rest of the row, and its block, as without it
    gen, nb = gen_for(5), 8
    c = torch.randn((1, T, 64), generator=gen).to(DT[dt])
    k = torch.randn((1, T, 16), generator=gen).to(DT[dt])
    bad = [(3, 7, float("nan")), (12, 0, float("inf")), (30, 63, float("-inf"))]
    c[0, 3, 7] = c[0, 12, 0] = c[0, 30, 63] = 0
    clean = gdla.qcache_empty(1, T, d_c=64, d_rope=16, scale_block=nb, device=DEV)
    gdla.qcache_write(*clean, c.to(DEV), k.to(DEV), scale_block=nb)
    for t, d, v in bad:
        c[0, t, d] = v
    k2 = k.clone()
    k2[0, 20, 5] = float("nan")
    dirty = gdla.qcache_empty(1, T, d_c=64, d_rope=16, scale_block=nb, device=DEV)
    gdla.qcache_write(*dirty, c.to(DEV), k2.to(DEV), scale_block=nb)
    mask = torch.zeros((T, 64), dtype=torch.bool)
    for t, d, _ in bad:
        mask[t, d] = True
    got, ref = dirty[0].float().cpu()[0], clean[0].float().cpu()[0]
    assert torch.isnan(got[mask]).all() and torch.equal(got[~mask], ref[~mask])
    got, ref = dirty[1].float().cpu()[0], clean[1].float().cpu()[0]
    assert torch.isnan(got[20, 5])
    got[20, 5] = ref[20, 5]
    assert torch.equal(got, ref)
    sc = f64(clean[2])[0]
    sc_d = f64(dirty[2])[0]
    keep = [b for b in range(T // nb) if b != 20 // nb]  # (the rotary value was a number before)
    assert (sc_d[keep] == sc[keep]).all()


def test_write_ranges_outside_the_cache_are_left_and_reported():
    T, L, d_c, d_r = 50, 10, 64, 16
    for start, lens in (([-1, 0], [5, 5]), ([45, 3], [6, 2]), ([0, 0], [11, 1]), ([0, 50], [-1, 0]), ([51, 0], [0, 10]),
                        ([2147483647, 0], [10, 10])):
        c8, kr8, sc = gdla.qcache_empty(2, T, d_c=d_c, d_rope=d_r, device=DEV)
        for t in (c8, kr8):
            t.view(torch.uint8).fill_(7)
        sc.fill_(3.0)
        c = torch.ones((2, L, d_c), device=DEV)
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        gdla.qcache_write(c8, kr8, sc, c, torch.ones((2, L, d_r), device=DEV), start=i32(start), lens=i32(lens),
                          workspace=ws)
        assert gdla.workspace_status(ws) == _abi.GDLA_ERR_INVALID_ARG
        for b in range(2):
            ok = 0 <= lens[b] <= L and 0 <= start[b] and start[b] + lens[b] <= T
            n = (c8.view(torch.uint8)[b] != 7).any(-1).sum()
            assert int(n) == (lens[b] if ok else 0), (start, lens, b)


# ------------------------------------------------------------------------- read
def made_cache(B, T, d_c, d_rope, nb, seed, spread=3):
    """Values of about one to 2^spread, quantised with each block's own scale."""
    gen = gen_for(seed)
    size = torch.exp2(torch.randint(0, spread + 1, (B, T, 1), generator=gen).float())
    c = torch.randn((B, T, d_c), generator=gen) * size
    k = torch.randn((B, T, d_rope), generator=gen) * size
    cache = gdla.qcache_empty(B, T, d_c=d_c, d_rope=d_rope, scale_block=nb, device=DEV)
    gdla.qcache_write(*cache, c.to(DEV), k.to(DEV), scale_block=nb)
    return cache


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("d_c,d_rope,T,first,L,nb,lens", [
    (512, 64, 300, 0, 300, 1, None), (512, 64, 300, 37, 200, 16, [200, 0, 1]), (256, 32, 129, 1, 128, 128, [5, 128, 127]),
    (64, 16, 1, 0, 1, 1, None), (128, 64, 70, 69, 1, 64, [1, 0, 1])])
def test_read(dt, d_c, d_rope, T, first, L, nb, lens):
    B = 3
    c8, kr8, sc = made_cache(B, T, d_c, d_rope, nb, seed=T)
    sc *= 1.37  # scales of the caller's own, not powers of two
    if lens is not None:  # rows that are not read hold anything
        for b in range(B):
            c8.view(torch.uint8)[b, first + lens[b]:] = 0x7F
            kr8.view(torch.uint8)[b, first + lens[b]:] = 0xFF
            blk = (first + lens[b] + nb - 1) // nb
            sc[b, blk:] = float("nan")
    c, k = gdla.qcache_read(c8, kr8, sc, length=L, first=first, lens=None if lens is None else i32(lens), scale_block=nb,
                            dtype=DT[dt])
    got = np.concatenate([f64(c), f64(k)], -1)
    ref = held(c8, kr8, sc, nb)[:, first:first + L]
    half = 2.0 ** -24 + (2.0 ** -8 if dt == "bf16" else 0.0)
    for b in range(B):
        n = L if lens is None else lens[b]
        assert (np.abs(got[b, :n] - ref[b, :n]) <= half * np.abs(ref[b, :n])).all()
        assert (got[b, n:] == 0).all()


def test_read_of_written_rows_is_exact_in_bf16():
    c8, kr8, sc = made_cache(2, 100, 512, 64, 16, seed=3)
    c, k = gdla.qcache_read(c8, kr8, sc, length=100, scale_block=16)
    assert (np.concatenate([f64(c), f64(k)], -1) == held(c8, kr8, sc, 16)).all()
    # the cache as plain bytes is the same cache
    c2, k2 = gdla.qcache_read(c8.view(torch.uint8), kr8.view(torch.uint8), sc, length=100, scale_block=16)
    assert torch.equal(c, c2) and torch.equal(k, k2)


@pytest.mark.parametrize("dt,d_c,d_rope,d_head,n_kv,T,first,L,nb,lens", [
    ("bf16", 512, 64, 128, 16, 333, 0, 333, 1, [333, 100]), ("bf16", 512, 64, 128, 3, 200, 64, 129, 16, [0, 129]),
    ("bf16", 512, 64, 128, 1, 1, 0, 1, 64, None), ("bf16", 256, 32, 64, 2, 150, 0, 150, 32, [149, 1]),
    ("fp32", 64, 16, 32, 4, 90, 10, 77, 8, [77, 3])])
def test_expand(dt, d_c, d_rope, d_head, n_kv, T, first, L, nb, lens):
    c8, kr8, sc = made_cache(2, T, d_c, d_rope, nb, seed=T + 1)
    w = (torch.randn((d_c, n_kv * 2 * d_head), generator=gen_for(9)) * d_c ** -0.5).to(DT[dt]).to(DEV)
    kv, kr, ch = gdla.qcache_expand(c8, kr8, sc, w, n_kv=n_kv, d_nope=d_head, d_v=d_head, length=L, first=first,
                                    lens=None if lens is None else i32(lens), scale_block=nb)
    ref = held(c8, kr8, sc, nb)[:, first:first + L]
    for b in range(2):
        if lens is not None:
            ref[b, lens[b]:] = 0
    assert (f64(ch) == ref[..., :d_c]).all() and (f64(kr) == ref[..., d_c:]).all()
    W = f64(w)
    want = ref[..., :d_c] @ W
    mag = np.abs(ref[..., :d_c]) @ np.abs(W)
    half = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    assert (np.abs(f64(kv).reshape(want.shape) - want) <= half * np.abs(want) + 2 * d_c * 2.0 ** -24 * mag).all()


# ----------------------------------------------------------------------- decode
def decode_inputs(B, T, n_kv, g, d_c, d_rope, d_head, dt, nb, lens, seed, spread=0, q_size=1.0):
    gen, dtype = gen_for(seed), DT[dt]
    H, S = n_kv * (g + 1), n_kv * g
    s = {"cache": made_cache(B, T, d_c, d_rope, nb, seed, spread), "nb": nb, "g": g, "d": d_head, "B": B}
    s["q"] = (torch.randn((B, H, d_head + d_rope), generator=gen) * q_size).to(dtype).to(DEV)
    s["w"] = (torch.randn((d_c, n_kv * 2 * d_head), generator=gen) * d_c ** -0.5).to(dtype).to(DEV)
    s["cos"], s["sin"] = gdla.rope_tables(T, d_rope, device=DEV)
    s["lam"] = torch.randn((B, S), generator=gen).to(DEV)
    s["gate"] = torch.randn((B, S, d_head), generator=gen).to(dtype).to(DEV)
    s["lens"] = lens
    return s


def call_decode(s, window=0, **kw):
    return gdla.qcache_decode(*s["cache"], s["q"], s["w"], s["cos"], s["sin"], s["lam"], s["gate"], i32(s["lens"]),
                              g=s["g"], scale_block=s["nb"], mask="sliding" if window else "causal", window=window, **kw)


def decode_ref(s, window=0):
    v = held(*s["cache"], s["nb"])
    d_c, out = s["cache"][0].shape[2], []
    for b, n in enumerate(s["lens"]):
        if n == 0:
            out.append(np.zeros(tuple(s["gate"].shape[1:])))
            continue
        lo = max(0, n - window) if window else 0
        rows = np.where((np.arange(n) >= lo)[:, None], v[b, :n], 0.0)
        out.append(oracle.decode_seq(c_hat=rows[:, :d_c].copy(), k_r_rot=rows[:, d_c:].copy(), q=f64(s["q"][b]),
                                     w_ukv=f64(s["w"]), lam=f64(s["lam"][b]), gate=f64(s["gate"][b]), g=s["g"],
                                     d_n=s["d"], d_v=s["d"], mask=mask_code("sliding" if window else "causal"),
                                     window=window))
    return np.stack(out)


def poison(s, window=0):
    """NaN rows and scales wherever the call may not look."""
    c8, kr8, sc = s["cache"]
    nb = s["nb"]
    for b, n in enumerate(s["lens"]):
        for sl in (slice(n, None), slice(0, max(0, n - window) if window else 0)):
            c8.view(torch.uint8)[b, sl] = 0x7F
            kr8.view(torch.uint8)[b, sl] = 0xFF
        sc[b, (n + nb - 1) // nb:] = float("nan")
        if window and n > window:
            sc[b, :(n - window) // nb] = float("nan")


R = dict(d_c=512, d_rope=64, d_head=128, dt="bf16")
DECODES = [
    # tensor-core path: tile borders, one token, empty slots, head groups, windows, scale blocks
    dict(R, B=1, T=1, n_kv=16, g=2, nb=1, lens=[1], window=0),
    dict(R, B=1, T=1500, n_kv=16, g=2, nb=64, lens=[1500], window=0),
    dict(R, B=5, T=300, n_kv=16, g=2, nb=1, lens=[300, 0, 1, 128, 129], window=0),
    dict(R, B=4, T=300, n_kv=16, g=2, nb=128, lens=[127, 255, 256, 257], window=0),
    dict(R, B=3, T=1000, n_kv=16, g=4, nb=16, lens=[1000, 513, 2], window=0),
    dict(R, B=3, T=1000, n_kv=16, g=3, nb=16, lens=[1000, 513, 77], window=100),
    dict(R, B=3, T=700, n_kv=16, g=5, nb=2, lens=[700, 700, 64], window=1),
    dict(R, B=2, T=520, n_kv=16, g=8, nb=32, lens=[520, 300], window=0),
    dict(R, B=7, T=257, n_kv=1, g=1, nb=1, lens=[257, 0, 0, 5, 200, 131, 0], window=128),
    dict(R, B=2, T=400, n_kv=3, g=2, nb=8, lens=[400, 399], window=129),
    dict(R, B=1, T=700, n_kv=49, g=1, nb=64, lens=[650], window=0),
    dict(R, B=200, T=130, n_kv=2, g=1, nb=64, lens=[(i * 37) % 131 for i in range(200)], window=0),
    dict(R, B=2, T=20000, n_kv=2, g=2, nb=64, lens=[20000, 11111], window=0),
    dict(R, B=4, T=30000, n_kv=1, g=3, nb=16, lens=[30000, 29000, 0, 27777], window=0),
    dict(R, B=3, T=30000, n_kv=2, g=1, nb=1, lens=[30000, 29000, 27777], window=25000),
    # CUDA cores: narrow widths, fp32
    dict(B=3, T=300, n_kv=2, g=3, d_c=256, d_rope=32, d_head=64, dt="bf16", nb=16, lens=[300, 0, 129], window=0),
    dict(B=3, T=300, n_kv=2, g=3, d_c=256, d_rope=32, d_head=64, dt="bf16", nb=1, lens=[300, 1, 129], window=50),
    dict(B=4, T=500, n_kv=4, g=2, d_c=64, d_rope=16, d_head=32, dt="fp32", nb=1, lens=[500, 0, 33, 1], window=0),
    dict(B=2, T=200, n_kv=16, g=3, d_c=512, d_rope=64, d_head=128, dt="fp32", nb=64, lens=[200, 90], window=65),
    dict(B=1, T=1, n_kv=1, g=1, d_c=128, d_rope=16, d_head=32, dt="fp32", nb=128, lens=[1], window=0),
]


@pytest.mark.parametrize("case", DECODES, ids=lambda c: f"{c['dt']}_B{c['B']}_T{c['T']}_kv{c['n_kv']}_g{c['g']}_nb{c['nb']}_w{c['window']}")
@pytest.mark.parametrize("spread", [0, 4])
def test_decode(case, spread):
    c = dict(case)
    window = c.pop("window")
    s = decode_inputs(**c, seed=c["T"] + c["g"], spread=spread)
    if spread:  # larger keys: keep the logits of ordinary size
        s["q"] = (s["q"].float() * 0.1).to(s["q"].dtype)
    ref = decode_ref(s, window)
    poison(s, window)
    need = gdla.qcache_decode_workspace_size(B=c["B"], T_max=c["T"], d_c=c["d_c"], d_rope=c["d_rope"], n_kv=c["n_kv"],
                                             d_nope=c["d_head"], d_v=c["d_head"], g=c["g"], dtype=DT[c["dt"]])
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)  # (NaN wherever nothing is written)
    y = call_decode(s, window, workspace=ws)
    assert gdla.workspace_status(ws) == _abi.GDLA_OK
    for b, n in enumerate(s["lens"]):
        if n == 0:
            assert (y[b] == 0).all()
    # an output may be a small difference of two heads: in fp32 the bar is absolute, and the
    # values grow with the spread
    size = 1.0 if c["dt"] == "bf16" else max(1.0, float(np.abs(ref).max()))
    assert_parity(f64(y) / size, ref / size, DT[c["dt"]], f"8-bit decode {c['dt']} T={c['T']} spread {spread}")
    # the same call again gives the same bits
    assert torch.equal(call_decode(s, window), y)


@pytest.mark.parametrize("B,T,n_kv,lens", [(2, 2000, 16, [2000, 1777]), (3, 40000, 2, [40000, 129, 33333])])
def test_decode_peaked_logits_and_rising_maxima(B, T, n_kv, lens):
    # logits up to ~100: one token carries the softmax, and the running maximum moves often
    # (the long case: shares of several tiles, two sequences in one share)
    s = decode_inputs(B, T, n_kv, 2, 512, 64, 128, "bf16", 1, lens, seed=77)
    s["q"] = (s["q"].float() * 6).to(torch.bfloat16)
    c8 = s["cache"][0]
    # rows that grow along the sequence
    t = torch.linspace(0, 1, T, device=DEV)[None, :, None]
    c8.copy_((c8.float() * (0.2 + 0.8 * t)).to(torch.float8_e4m3fn))
    ref = decode_ref(s)
    # (as for the bf16 cache: operands of 8 bits move a logit of size s by about s 2^-8)
    v = held(*s["cache"], 1)
    top = 0.0
    W, q = f64(s["w"]).reshape(512, n_kv, 256), f64(s["q"])
    for b, n in enumerate(s["lens"]):
        for h in range(n_kv):
            ql = q[b, 2 * h, :128] @ W[:, h, :128].T
            top = max(top, float(np.abs(v[b, :n, :512] @ ql).max()) / np.sqrt(192))
    assert_parity(f64(call_decode(s)), ref, torch.bfloat16, "8-bit decode, peaked", elem_bound=0.1 + 8 * top * 2.0 ** -8)


def test_decode_zero_rows_among_others():
    # rows of zeros have the smallest scale, 2^-40, next to scales of ordinary size
    s = decode_inputs(2, 600, 16, 2, 512, 64, 128, "bf16", 1, [600, 333], seed=12)
    for b in range(2):
        sel = torch.arange(0, 600, 3, device=DEV)
        s["cache"][0].view(torch.uint8)[b, sel] = 0
        s["cache"][1].view(torch.uint8)[b, sel] = 0
        s["cache"][2][b, sel] = 2.0 ** -40
    assert_parity(f64(call_decode(s)), decode_ref(s), torch.bfloat16, "8-bit decode, zero rows")
    # nothing but zero rows: equal weights over zeros
    for t in s["cache"][:2]:
        t.view(torch.uint8).zero_()
    s["cache"][2].fill_(2.0 ** -40)
    assert (call_decode(s) == 0).all()


def test_decode_passes_on_a_nan_that_it_sees():
    for dt, dims in (("bf16", (16, 2, 512, 64, 128)), ("fp32", (4, 2, 64, 16, 32))):
        s = decode_inputs(3, 400, dims[0], dims[1], *dims[2:], dt, 1, [400, 300, 200], seed=8)
        clean = call_decode(s)
        s["cache"][0].view(torch.uint8)[1, 170, 5] = 0x7F
        y = call_decode(s)
        assert torch.isnan(y[1]).all()
        assert torch.equal(y[0], clean[0]) and torch.equal(y[2], clean[2])


def test_decode_lengths_outside_the_cache_are_clamped_and_reported():
    s = decode_inputs(3, 200, 16, 2, 512, 64, 128, "bf16", 1, [200, 0, 50], seed=4)
    ref = call_decode(s)
    s["lens"] = [5000, -3, 50]
    ws = torch.zeros(gdla.qcache_decode_workspace_size(B=3, T_max=200, d_c=512, d_rope=64, n_kv=16, d_nope=128, d_v=128,
                                                       g=2), dtype=torch.uint8, device=DEV)
    y = call_decode(s, workspace=ws)
    assert gdla.workspace_status(ws) == _abi.GDLA_ERR_INVALID_ARG
    assert torch.equal(y, ref)


def test_decode_of_a_batch_with_nothing_in_it():
    for dt, dims in (("bf16", (16, 2, 512, 64, 128)), ("fp32", (4, 2, 64, 16, 32))):
        s = decode_inputs(4, 300, dims[0], dims[1], *dims[2:], dt, 1, [0, 0, 0, 0], seed=6)
        poison(s)
        for _ in range(3):
            assert (call_decode(s) == 0).all()


def test_decode_agrees_with_the_bf16_cache():
    # the 8-bit values are exact in bf16, so both caches hold the same numbers
    s = decode_inputs(4, 3000, 16, 2, 512, 64, 128, "bf16", 64, [3000, 1, 2048, 999], seed=21)
    c, k = gdla.qcache_read(*s["cache"], length=3000, scale_block=64)
    y16 = gdla.decode(c, k, s["q"], s["w"], s["cos"], s["sin"], s["lam"], s["gate"], i32(s["lens"]), g=2)
    y8 = call_decode(s)
    assert_parity(f64(y8), f64(y16), torch.bfloat16, "8-bit decode against the bf16 cache")


# ------------------------------------------------------------------- as it is used
def test_prompt_in_chunks_then_steps():
    """A prompt prefilled in chunks over the 8-bit cache, and decode steps behind it: every
    chunk and step attends over what the cache holds."""
    n_kv, g, T, B = 2, 2, 700, 2
    shape = wl.PrefillShape("chunks", B=B, L=T, n_kv=n_kv, g=g)
    inp = wl.make_prefill_inputs(shape, seed=5, device=DEV)
    cos, sin = gdla.rope_tables(T, 64, device=DEV)
    nb = 32
    cache = gdla.qcache_empty(B, T, scale_block=nb, device=DEV)
    for t in cache[:2]:
        t.view(torch.uint8).fill_(0x7F)
    at = 0

    def write(n):
        sl = slice(at, at + n)
        gdla.qcache_write(*cache, inp["c_kv"][:, sl].contiguous(), inp["k_rope"][:, sl].contiguous(), gamma=inp["gamma"],
                          rope_cos=cos, rope_sin=sin, start=i32([at] * B), scale_block=nb)

    def rows(name, i0, i1):
        return inp[name][:, i0:i1].clone(memory_format=torch.contiguous_format)

    def reference(upto, i0):
        v = held(*cache, nb)[:, :upto]
        out = []
        for b in range(B):
            for i in range(i0, upto):
                q = f64(inp["q"][b, i])
                out.append(oracle.decode_seq(c_hat=v[b, :i + 1, :512].copy(), k_r_rot=v[b, :i + 1, 512:].copy(), q=q,
                                             w_ukv=f64(inp["w_ukv"]), lam=f64(inp["lam_logits"][b, i]),
                                             gate=f64(inp["gate_logits"][b, i]), g=g, d_n=128, d_v=128,
                                             mask=mask_code("causal"), window=0))
        return np.stack(out)

    for n in (300, 133, 1, 200):
        write(n)
        kv, kr, _ = gdla.qcache_expand(*cache, inp["w_ukv"], n_kv=n_kv, d_nope=128, d_v=128, length=at + n, scale_block=nb)
        y = gdla.attend(rows("q", at, at + n), kv, kr, cos, sin, rows("lam_logits", at, at + n),
                        rows("gate_logits", at, at + n), g=g, q_start=at)
        assert_parity(f64(y).reshape(-1, n_kv * g, 128), reference(at + n, at), torch.bfloat16, f"chunk at {at}")
        at += n
    for _ in range(20):
        write(1)
        i = at
        at += 1
        y = gdla.qcache_decode(*cache, inp["q"][:, i].contiguous(), inp["w_ukv"], cos, sin,
                               inp["lam_logits"][:, i].contiguous(), inp["gate_logits"][:, i].contiguous(),
                               i32([at] * B), g=g, scale_block=nb)
        assert_parity(f64(y), reference(at, i), torch.bfloat16, f"step {i}")
    # and the whole is near the exact attention: e4m3 rows move it by a few per cent
    ref = oracle_prefill_rows(inp, [(b, at - 1) for b in range(B)], g=g, d_nope=128, d_v=128)
    e = f64(y) - ref
    assert np.sqrt((e * e).mean()) <= 0.2 * np.sqrt((ref * ref).mean())


def test_quantising_a_prefill_cache():
    # prefill's own bf16 cache outputs, taken over as rows that are normalised already
    shape = wl.PrefillShape("take over", B=2, L=150, n_kv=2, g=2)
    inp = wl.make_prefill_inputs(shape, seed=6, device=DEV)
    cos, sin = gdla.rope_tables(shape.L, 64, device=DEV)
    kv, kr, ch = gdla.latent_expand(inp["c_kv"], inp["gamma"], inp["k_rope"], inp["w_ukv"], cos, sin, n_kv=2, d_nope=128,
                                    d_v=128)
    cache = gdla.qcache_empty(2, 200, scale_block=1, device=DEV)
    gdla.qcache_write(*cache, ch, kr)
    x = np.concatenate([f64(ch), f64(kr)], -1)
    s = f64(cache[2])[:, :150, None]
    assert (s[..., 0] == np.vectorize(scale_of)(np.abs(x).max(-1))).all()
    assert_quantised(np.concatenate([e4m3_values(cache[0]), e4m3_values(cache[1])], -1)[:, :150], x, s)


def test_captured_and_replayed_step():
    B, T, n_kv, g, nb = 4, 500, 16, 2, 16
    s = decode_inputs(B, T, n_kv, g, 512, 64, 128, "bf16", nb, [100, 200, 300, 17], seed=31)
    gen = gen_for(32)
    c_kv = torch.randn((B, 1, 512), generator=gen).bfloat16().to(DEV)
    k_rope = torch.randn((B, 1, 64), generator=gen).bfloat16().to(DEV)
    gamma = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    start, lens = i32(s["lens"]), i32([n + 1 for n in s["lens"]])
    ws = torch.empty(gdla.qcache_decode_workspace_size(B=B, T_max=T, d_c=512, d_rope=64, n_kv=n_kv, d_nope=128, d_v=128,
                                                       g=g), dtype=torch.uint8, device=DEV)
    ws_w = torch.empty(256, dtype=torch.uint8, device=DEV)
    out = torch.empty((B, n_kv * g, 128), dtype=torch.bfloat16, device=DEV)

    def step(cache, y):
        gdla.qcache_write(*cache, c_kv, k_rope, gamma=gamma, rope_cos=s["cos"], rope_sin=s["sin"], start=start,
                          scale_block=nb, workspace=ws_w)
        gdla.qcache_decode(*cache, s["q"], s["w"], s["cos"], s["sin"], s["lam"], s["gate"], lens, g=g, scale_block=nb,
                           out=y, workspace=ws)

    eager = [t.clone() for t in s["cache"]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    warm = [t.clone() for t in s["cache"]]
    with torch.cuda.stream(side):
        step(warm, out)
        side.synchronize()
        graph.capture_begin()
        step(s["cache"], out)
        graph.capture_end()
    torch.cuda.current_stream().wait_stream(side)
    for i in range(5):
        # new inputs in the same buffers
        c_kv.copy_(torch.randn((B, 1, 512), generator=gen))
        k_rope.copy_(torch.randn((B, 1, 64), generator=gen))
        s["q"].copy_(torch.randn(s["q"].shape, generator=gen))
        out.fill_(float("nan"))
        graph.replay()
        want = torch.empty_like(out)
        torch.cuda.synchronize()
        step(eager, want)
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        for a, b in zip(s["cache"], eager):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        start += 1
        lens += 1
    assert gdla.workspace_status(ws) == _abi.GDLA_OK


def test_calls_on_two_streams_at_once():
    ss = [decode_inputs(8, 2000, 16, 2, 512, 64, 128, "bf16", 1, [2000 - 100 * i - j for i in range(8)], seed=40 + j)
          for j in range(2)]
    want = [call_decode(s) for s in ss]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ss]
    got = [[], []]
    for _ in range(10):
        for j, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[j].append(call_decode(ss[j]))
    # the stream as an argument, while another one is current
    other = [call_decode(s, stream=st, out=torch.empty_like(w), workspace=torch.empty(
        gdla.qcache_decode_workspace_size(B=8, T_max=2000, d_c=512, d_rope=64, n_kv=16, d_nope=128, d_v=128, g=2),
        dtype=torch.uint8, device=DEV)) for s, st, w in zip(ss, streams, want)]
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(y, want[j]) for y in got[j])
        assert torch.equal(other[j], want[j])


def test_offsets_past_32_bits():
    # 9 sequences of 2^20 tokens: the last ones begin past 2^32 bytes of the cache
    B, T = 9, 1 << 20
    c8, kr8, sc = gdla.qcache_empty(B, T, device=DEV)
    c8.view(torch.uint8).fill_(0x7F)
    kr8.view(torch.uint8).fill_(0x7F)
    sc.fill_(float("nan"))
    gen, L, w = gen_for(50), 130, 100
    c = torch.randn((B, L, 512), generator=gen).bfloat16().to(DEV)
    k = torch.randn((B, L, 64), generator=gen).bfloat16().to(DEV)
    start = [T - L - b for b in range(B)]
    gdla.qcache_write(c8, kr8, sc, c, k, start=i32(start))
    small = gdla.qcache_empty(B, L, device=DEV)
    gdla.qcache_write(*small, c, k)
    got = gdla.qcache_read(c8, kr8, sc, length=L, first=T - L - B + 1)
    for b in range(B):
        o = B - 1 - b
        n = L - o
        assert torch.equal(got[0][b, o:], small[0][b, :n].float().mul(small[2][b, :n, None]).bfloat16())
        assert torch.equal(got[1][b, o:], small[1][b, :n].float().mul(small[2][b, :n, None]).bfloat16())
    s = decode_inputs(B, 200, 16, 2, 512, 64, 128, "bf16", 1, [L] * B, seed=51)
    s["cache"] = small
    cos = torch.ones((T, 32), device=DEV)
    sin = torch.zeros((T, 32), device=DEV)  # (the same rotation, none, at both positions)
    y = gdla.qcache_decode(c8, kr8, sc, s["q"], s["w"], cos, sin, s["lam"], s["gate"], i32([T - b for b in range(B)]), g=2,
                           mask="sliding", window=w)
    ref = gdla.qcache_decode(*small, s["q"], s["w"], cos[:L].contiguous(), sin[:L].contiguous(), s["lam"], s["gate"],
                             i32([L] * B), g=2, mask="sliding", window=w)
    assert_parity(f64(y), f64(ref), torch.bfloat16, "8-bit decode past 2^32 bytes")


def test_refusals_on_the_device():
    c8, kr8, sc = gdla.qcache_empty(2, 64, device=DEV)
    c = torch.zeros((2, 8, 512), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((2, 8, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        gdla.qcache_write(c8, kr8, sc, c.transpose(0, 1).contiguous().transpose(0, 1), k)
    with pytest.raises(gdla.GdlaError):
        gdla.qcache_write(c8, kr8, sc, c, k, workspace=torch.zeros(128, dtype=torch.uint8, device=DEV))
    with pytest.raises(gdla.GdlaError):
        gdla.qcache_read(c8, kr8, sc, length=64, first=1)
    with pytest.raises(ValueError):
        gdla.qcache_read(c8, kr8, sc[:1], length=64)


# ------------------------------------------------------- a sink over a flat tail
def sink_inputs(T, n_kv, g, nb, gap, sinks, size, B=1, seed=70):
    """Sequences whose sink tokens score ``gap`` powers of two above all the others, which are
    nearly flat and share a common component; the sinks' own latents are ``size`` of theirs.
    The gap comes from two rotary columns whose products are exact in every operand type
    (tau log2e is 2^-4, the tables rotate by nothing), so that no rounding of a score moves it."""
    s = decode_inputs(B, T, n_kv, g, 512, 64, 128, "bf16", nb, [T] * B, seed, q_size=0.25)
    gen = gen_for(seed + 1)
    c = 1.0 + torch.randn((B, T, 512), generator=gen)
    k = torch.zeros((B, T, 64))
    whole = int(gap) // 2 * 2
    for b in range(B):
        c[b, sinks] *= size
        k[b, sinks, 0], k[b, sinks, 1] = float(whole), (gap - whole) * 16
    gdla.qcache_write(*s["cache"], c.to(DEV), k.to(DEV), scale_block=nb)
    s["q"][..., 128:] = 0
    s["q"][..., 128], s["q"][..., 129] = 16.0, 1.0
    s["cos"], s["sin"] = torch.ones_like(s["cos"]), torch.zeros_like(s["sin"])
    s["tau"] = float(np.log(2.0)) / 16
    return s


def sink_ref(s, window=0, kv_sel=None):
    v = held(*s["cache"], s["nb"])
    return np.stack([oracle.decode_seq(c_hat=v[b, :n, :512].copy(), k_r_rot=v[b, :n, 512:].copy(), q=f64(s["q"][b]),
                                       w_ukv=f64(s["w"]), lam=f64(s["lam"][b]), gate=f64(s["gate"][b]), g=s["g"],
                                       d_n=128, d_v=128, mask=mask_code("sliding" if window else "causal"),
                                       window=window, scale=s["tau"], inv_freq=np.zeros(32), kv_sel=kv_sel)
                     for b, n in enumerate(s["lens"])])


# a share of one tile, of some, and of 14336 tokens (24 head groups: 6 shares of the cache)
SINKS = [
    dict(T=128, n_kv=2, g=2, nb=64, sinks=[0]),
    dict(T=97, n_kv=2, g=2, nb=16, sinks=[96]),
    dict(T=1500, n_kv=16, g=2, nb=1, sinks=[3]),
    dict(T=1500, n_kv=16, g=2, nb=64, sinks=[0, 1, 2, 700, 1400]),
    dict(T=2000, n_kv=16, g=4, nb=128, sinks=list(range(300, 316))),
    dict(T=40000, n_kv=2, g=2, nb=64, sinks=[39999]),
    dict(T=86016, n_kv=128, g=8, nb=64, sinks=[0]),
]


@pytest.mark.parametrize("case", SINKS, ids=lambda c: f"T{c['T']}_kv{c['n_kv']}_g{c['g']}_nb{c['nb']}_n{len(c['sinks'])}")
@pytest.mark.parametrize("gap", [12.0, 18.0, 19.5, 20.0, 21.0, 30.0])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -8, 1.0])
def test_decode_sink_over_a_flat_tail(case, gap, size):
    # each other token weighs next to nothing, all of them together do not: the parity bar as it
    # is, for the 8-bit and the bf16 cache of the same values
    s = sink_inputs(**case, gap=gap, size=size)
    sel = [0, case["n_kv"] - 1] if case["n_kv"] > 16 else None
    ref = sink_ref(s, kv_sel=sel)
    y = call_decode(s, softmax_scale=s["tau"])
    assert_parity(f64(y), ref, torch.bfloat16, f"8-bit decode, sink {gap} {size} T={case['T']}")
    c, k = gdla.qcache_read(*s["cache"], length=case["T"], scale_block=case["nb"])
    y16 = gdla.decode(c, k, s["q"], s["w"], s["cos"], s["sin"], s["lam"], s["gate"], i32(s["lens"]), g=case["g"],
                      softmax_scale=s["tau"])
    assert_parity(f64(y16), ref, torch.bfloat16, f"bf16 decode, sink {gap} {size} T={case['T']}")


@pytest.mark.parametrize("gap", [16.0, 18.0, 20.0])
def test_decode_long_tail_behind_many_large_weights(gap):
    # 40 tokens of the first tile, of small values, carry most of the softmax: the reference is
    # theirs until it follows the tail, 8 of the 112 tiles of the first share at most
    s = sink_inputs(86016, 128, 8, 64, gap, list(range(40)), 2.0 ** -6, seed=72)
    ref = sink_ref(s, kv_sel=[0, 127])
    assert_parity(f64(call_decode(s, softmax_scale=s["tau"])), ref, torch.bfloat16, f"8-bit decode, 40 sinks {gap}")


@pytest.mark.parametrize("q_size", [0.5, 2.0, 4.0, 8.0])
@pytest.mark.parametrize("T,lens", [(9000, [9000, 8000]), (700, [700, 129])])
def test_decode_broad_softmax(T, lens, q_size):
    # logits of half a nat to eight of deviation: the reference rises often, and the tiles are
    # looked at; a logit of size s moves by s 2^-8 (the query's two 8-bit terms)
    s = decode_inputs(2, T, 3, 2, 512, 64, 128, "bf16", 16, lens, seed=73, q_size=q_size)
    ref = decode_ref(s)
    assert_parity(f64(call_decode(s)), ref, torch.bfloat16, f"8-bit decode, logits x {q_size}",
                  elem_bound=0.1 + 8 * (5 * q_size) * 2.0 ** -8)


@pytest.mark.parametrize("window", [0, 700])
def test_decode_sinks_in_a_batch(window):
    # sinks inside and in front of the window, at tile borders; several sequences in one share
    s = sink_inputs(900, 2, 1, 64, 20.0, [0, 127, 128, 500, 899], 0.0, B=60, seed=71)
    s["lens"] = [900 - 13 * (i % 7) for i in range(60)]
    ref = sink_ref(s, window)
    poison(s, window)
    y = call_decode(s, window, softmax_scale=s["tau"])
    assert_parity(f64(y), ref, torch.bfloat16, f"8-bit decode, sinks in a batch, window {window}")
    assert torch.equal(call_decode(s, window, softmax_scale=s["tau"]), y)


# ------------------------------------------------------- what a workspace held before
STALE = [_abi.GDLA_ERR_TIMEOUT, _abi.GDLA_ERR_CUDA, _abi.GDLA_ERR_INVALID_ARG, -1]


@pytest.mark.parametrize("code", STALE)
def test_decode_in_a_workspace_of_a_failed_call(code):
    # the status word of the call before, and every other word, say nothing to this one: the query
    # images are written whatever they hold
    for B, n_kv, g in ((3, 16, 2), (200, 16, 4)):
        s = decode_inputs(B, 140, n_kv, g, 512, 64, 128, "bf16", 1, [1 + (37 * b) % 140 for b in range(B)], seed=80)
        want = call_decode(s)
        need = gdla.qcache_decode_workspace_size(B=B, T_max=140, d_c=512, d_rope=64, n_kv=n_kv, d_nope=128, d_v=128, g=g)
        ws = torch.empty(need // 4, dtype=torch.int32, device=DEV)
        for _ in range(10):
            ws.fill_(code)
            y = call_decode(s, workspace=ws)
            assert gdla.workspace_status(ws) == _abi.GDLA_OK
            assert torch.equal(y, want)


@pytest.mark.parametrize("code", STALE)
@pytest.mark.parametrize("L", [1, 300, 6000])
def test_write_in_a_workspace_of_a_failed_call(code, L):
    gen = gen_for(81)
    c = torch.randn((3, L, 512), generator=gen).bfloat16().to(DEV)
    k = torch.randn((3, L, 64), generator=gen).bfloat16().to(DEV)
    want = gdla.qcache_empty(3, L, scale_block=16, device=DEV)
    gdla.qcache_write(*want, c, k, scale_block=16)
    ws = torch.empty(64, dtype=torch.int32, device=DEV)
    for _ in range(10):
        got = gdla.qcache_empty(3, L, scale_block=16, device=DEV)
        for t in got:
            t.view(torch.uint8).fill_(0x55)
        ws.fill_(code)
        gdla.qcache_write(*got, c, k, scale_block=16, workspace=ws)
        assert gdla.workspace_status(ws) == _abi.GDLA_OK
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    # a range that does not fit is reported whatever the word held
    ws.fill_(code)
    gdla.qcache_write(*got, c, k, scale_block=16, lens=i32([L, L, L]), start=i32([0, 1, 0]), workspace=ws)
    assert gdla.workspace_status(ws) == _abi.GDLA_ERR_INVALID_ARG


@pytest.mark.parametrize("dt,L", [("bf16", 5), ("fp32", 5), ("bf16", 17000)])
def test_write_maxima_past_fp32(dt, L):
    # a normalised latent past fp32's range (one element of many, a large gain): its block takes
    # the scale that it needs, and what is stored is its value over that
    gen = gen_for(82)
    c = 0.01 * torch.randn((1, L, 64), generator=gen)
    c[0, 1::2] = 0
    c[0, 1::2, 7] = 0.16
    c = c.to(DT[dt])
    gamma = torch.ones(64).to(DT[dt])
    gamma[7] = 3e38
    cos, sin = gdla.rope_tables(L, 16, device=DEV)
    cache = gdla.qcache_empty(1, L, d_c=64, d_rope=16, device=DEV)
    gdla.qcache_write(*cache, c.to(DEV), torch.zeros((1, L, 16), dtype=DT[dt], device=DEV), gamma=gamma.to(DEV),
                      rope_cos=cos, rope_sin=sin)
    x = f64(c)[0]
    x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * f64(gamma)
    top = np.abs(x).max(-1)
    assert top[1] > 2.0 ** 128 and top[0] > 0
    e = np.frexp(top / 448)
    want = np.maximum(np.where(e[0] == 0.5, np.exp2(e[1] - 1.0), np.exp2(e[1] * 1.0)), 2.0 ** -40)
    assert (f64(cache[2])[0] == want).all()
    assert_quantised(e4m3_values(cache[0])[0], x, want[:, None])


@pytest.mark.parametrize("handle", [False, True])
def test_defaults_on_a_given_stream(handle):
    # What a call allocates by itself is its stream's. The given stream is held up, so that the call's
    # kernels run after the current stream has taken and filled memory of the same sizes; and the
    # current stream is, so that it still writes to memory that was freed before the call.
    B, T = 4, 600
    s = decode_inputs(B, T, 16, 2, 512, 64, 128, "bf16", 16, [600, 1, 300, 77], seed=90)
    c_kv = torch.randn((B, T, 512), generator=gen_for(91)).bfloat16().to(DEV)
    k_rope = torch.randn((B, T, 64), generator=gen_for(92)).bfloat16().to(DEV)
    need = gdla.qcache_decode_workspace_size(B=B, T_max=T, d_c=512, d_rope=64, n_kv=16, d_nope=128, d_v=128, g=2)
    side = torch.cuda.Stream()
    lens = i32(s["lens"])

    def calls(stream):
        cache = [t.clone() for t in s["cache"]]
        torch.cuda.synchronize()
        kw = {} if stream is None else {"stream": stream.cuda_stream if handle else stream}
        for st in (stream, torch.cuda.current_stream()) if stream is not None else ():
            with torch.cuda.stream(st):
                torch.cuda._sleep(40_000_000)
        sizes = (256, need, B * 32 * 128 * 2, B * T * 512 * 2, B * T * 64 * 2, B * T * 16 * 256 * 2)
        freed = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
        for t in freed:
            t.fill_(0xFF)
        del freed, t
        gdla.qcache_write(*cache, c_kv, k_rope, scale_block=16, **kw)
        out = [gdla.qcache_decode(*cache, s["q"], s["w"], s["cos"], s["sin"], s["lam"], s["gate"], lens, g=2,
                                  scale_block=16, **kw)]
        out += gdla.qcache_read(*cache, length=T, scale_block=16, **kw)
        out += gdla.qcache_expand(*cache, s["w"], n_kv=16, d_nope=128, d_v=128, length=T, scale_block=16, **kw)
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(2)]
        torch.cuda.synchronize()
        del junk
        return out

    want = calls(None)
    assert all(torch.isfinite(t.float()).all() for t in want)
    for got, ref in zip(calls(side), want):
        assert torch.equal(got, ref)


# head groups of up to 16, 32 and 48 heads, full and padded, with sinks and without
@pytest.mark.parametrize("n_kv,g", [(16, 1), (5, 4), (4, 3), (7, 1), (16, 3), (16, 4)])
@pytest.mark.parametrize("gap", [0.0, 20.0])
@pytest.mark.parametrize("nb", [1, 64])
def test_decode_head_groups(n_kv, g, gap, nb):
    s = sink_inputs(1100, n_kv, g, nb, gap, [0, 600, 601], 2.0 ** -4, B=2, seed=95)
    s["lens"] = [1100, 650]
    ref = sink_ref(s)
    y = call_decode(s, softmax_scale=s["tau"])
    assert_parity(f64(y), ref, torch.bfloat16, f"8-bit decode, {n_kv * (g + 1)} heads, sink {gap}")
    # a share of several tiles gives what the same sequence alone gives, in one tile a share
    many = {**s, "cache": [t[:1].expand(70, *t.shape[1:]).contiguous() for t in s["cache"]],
            **{n: s[n][:1].expand(70, *s[n].shape[1:]).contiguous() for n in ("q", "lam", "gate")}, "lens": [1100] * 70}
    ym = call_decode(many, softmax_scale=s["tau"])
    for b in (0, 33, 69):
        assert_parity(f64(ym[b]), ref[0], torch.bfloat16, f"8-bit decode, {n_kv * (g + 1)} heads, one of 70")


@pytest.mark.parametrize("levels", [
    [(40, [0], 0.0), (18, list(range(5, 17)), 0.125)],                                  # few behind a sink, and no crowd
    [(24, list(range(60)), 0.0)],                                                       # half a tile of sinks
    [(32, [0, 130, 131, 300], 0.0), (24, list(range(140, 180)), 2.0 ** -6)],
    [(16, list(range(0, 400, 50)), 0.0), (30, [399], 0.0)],
])
@pytest.mark.parametrize("T", [320, 400])
def test_decode_levels(levels, T):
    # tokens at several heights above the others
    s = sink_inputs(T, 5, 4, 128, 0.0, [], 1.0, seed=96)
    gen = gen_for(97)
    c, k = 1.0 + torch.randn((1, T, 512), generator=gen), torch.zeros((1, T, 64))
    for gap, tokens, size in levels:
        tokens = [t for t in tokens if t < T]
        c[0, tokens] *= size
        k[0, tokens, 0] = float(gap)
    gdla.qcache_write(*s["cache"], c.to(DEV), k.to(DEV), scale_block=128)
    y = call_decode(s, softmax_scale=s["tau"])
    assert_parity(f64(y), sink_ref(s), torch.bfloat16, f"8-bit decode, levels {[g for g, *_ in levels]}")


def test_allocations_are_the_given_streams():
    c8, kr8, sc = made_cache(2, 700, 512, 64, 16, seed=98)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream, want in ((side, side.cuda_stream), (side.cuda_stream, side.cuda_stream), (0, 0), (1, 0),
                         (torch.cuda.default_stream(), 0)):
        for current in (torch.cuda.default_stream(), torch.cuda.Stream()):
            with torch.cuda.stream(current):
                out = gdla.qcache_read(c8, kr8, sc, length=700, scale_block=16, stream=stream)
            torch.cuda.synchronize()
            for t in out:
                at = [g for g in torch.cuda.memory_snapshot() if g["address"] <= t.data_ptr() < g["address"] + g["total_size"]]
                assert [g["stream"] for g in at] == [want]
            assert (np.concatenate([f64(t) for t in out], -1) == held(c8, kr8, sc, 16)).all()
