"""Parity of the norm, rotation and cache write (CUDA, through the C ABI) with the fp64 oracle.

Tolerances, from the arithmetic: rows are normed in fp32 (a sum of up to 1024
squares in 32 partial sums, one square root, one division, one product: below
50 roundings of 2^-24, 3e-6 of the element before the bias), the angle is
formed in 64 bits and its sine and cosine are off by less than 3e-7, the
rotation adds two products: an element is within 5e-6 of the largest magnitude
among its pair and its parts of the fp64 one, checked against 1e-5 of the
row's largest magnitude.  A bf16 output adds half a step (2^-8 of itself); an
fp8 one half an e4m3 step (2^-4 of itself, or 2^-10, half the smallest
subnormal step, of the scale).  An fp8 row's scale is the fp32 quotient of its
largest magnitude by 448: 1e-5 of itself.
"""

import numpy as np
import pytest
import torch

from oracle.attention import norm_rope

pytestmark = pytest.mark.gpu

FINE = 1e-5


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_indexer_lightning_b200 import build as b
    b.build()
    import sparse_attention_indexer_lightning_b200 as lib
    return lib


def make(T, Hq, Hk, d, rope, norm_dim, seed, pos_max=100000):
    g = torch.Generator().manual_seed(seed)
    qk = (torch.randn(T, (Hq + Hk) * d + 16, generator=g) * 3 + 0.5).to(torch.bfloat16).cuda()
    f = lambda: torch.randn(norm_dim, generator=g).cuda()  # noqa: E731
    return dict(q=qk[:, :Hq * d].unflatten(1, (Hq, d)), k=qk[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d)),
                pos=torch.randint(0, pos_max, (T,), generator=g).cuda(),
                inv_freq=(10000.0 ** (-torch.arange(0, rope, 2).double() / max(rope, 1))).float().cuda(),
                qw=1 + 0.3 * f(), qb=0.3 * f(), kw=1 + 0.3 * f(), kb=0.3 * f())


def check(got, scale, ref, what):
    got, top = got.double().cpu().numpy(), np.abs(ref).max(axis=-1, keepdims=True)
    if scale is None:
        tol = FINE * top + 2.0 ** -8 * np.abs(ref) * (1 + FINE)
    else:
        s = scale.double().cpu().numpy().reshape(top.shape)
        want = np.where(top > 0, top / 448.0, 1.0)
        assert np.all(np.abs(s - want) <= FINE * want), f"{what}: scales"
        got = got * s
        tol = 2 * FINE * top + np.maximum(2.0 ** -4 * np.abs(ref) * (1 + FINE), 2.0 ** -10 * want)
    err = np.abs(got - ref)
    assert np.all(err <= tol), f"{what}: {np.max(err - tol):.3e} over the bound"


CASES = [
    # T, Hq, Hk, d, rope, rope_off, norm_dim, q norm, k norm, interleaved
    (1, 1, 1, 128, 64, 0, 128, "rms", "layer", False),
    (5, 32, 1, 128, 64, 0, 128, "none", "layer", False),
    (3, 32, 1, 128, 64, 64, 128, "rms", "layer", True),
    (7, 128, 1, 576, 64, 512, 512, "none", "rms", True),
    (2, 3, 2, 64, 64, 0, 64, "layer", "rms", False),
    (2, 3, 2, 8, 2, 6, 8, "layer", "rms", True),
    (4, 2, 1, 1024, 256, 768, 1024, "rms", "layer", False),
    (4, 9, 4, 200, 30, 101, 104, "rms", "layer", False),
    (4, 9, 4, 200, 30, 101, 104, "layer", "none", True),
    (300, 8, 1, 192, 0, 0, 192, "rms", "rms", False),
    (1000, 1, 1, 256, 128, 1, 256, "rms", "rms", False),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_norm_rope(L, case, fp8):
    T, Hq, Hk, d, rope, off, nd, qn, kn, inter = case
    s = make(T, Hq, Hk, d, rope, nd, seed=d + T)
    qw, qb = (s["qw"], s["qb"]) if qn != "none" else (None, None)
    kw, kb = (s["kw"], s["kb"]) if kn != "none" else (None, None)
    out = L.ls_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"] if rope else None, q_norm=qn, k_norm=kn, norm_dim=nd,
                         q_weight=qw, q_bias=qb, k_weight=kw, k_bias=kb, eps=1e-5, rope_off=off, interleaved=inter,
                         fp8=fp8)
    c = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    for x, norm, w, b, y, sc, name in ((s["q"], qn, qw, qb, out[0], out[1], "q"),
                                       (s["k"], kn, kw, kb, out[2], out[3], "k")):
        ref = norm_rope(c(x), c(s["pos"]), c(s["inv_freq"])[:rope // 2], norm, nd, c(w), c(b), 1e-5, off, inter)
        check(y, sc, ref, name)


@pytest.mark.parametrize("fp8", [False, True])
def test_cache_slots(L, fp8):
    """Keys go to the rows their slots name (-1: nowhere), and no other row of the cache changes."""
    T, d, R = 50, 128, 400
    s = make(T, 4, 1, d, 64, d, seed=2)
    g = torch.Generator().manual_seed(3)
    slots = torch.randperm(R, generator=g)[:T].cuda()
    slots[[3, 17]] = -1
    cache = torch.randn(R, d, generator=g).cuda().to(torch.float8_e4m3fn if fp8 else torch.bfloat16)
    scale = torch.rand(R, generator=g).cuda() if fp8 else None
    before, sb = cache.view(torch.uint8).clone(), None if scale is None else scale.clone()
    _, _, want, ws = L.ls_norm_rope(None, s["k"], s["pos"], s["inv_freq"], k_norm="rms", fp8=fp8)
    q, qs, k, ks = L.ls_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], k_norm="rms", k_cache=cache, k_scale=scale,
                                  slots=slots)
    assert k is cache and ks is scale and (qs is not None) == fp8
    on = slots >= 0
    assert torch.equal(cache.view(torch.uint8)[slots[on]], want.view(torch.uint8)[on, 0])
    rest = torch.ones(R, dtype=torch.bool, device="cuda")
    rest[slots[on]] = False
    assert torch.equal(cache.view(torch.uint8)[rest], before[rest])
    if fp8:
        assert torch.equal(scale[slots[on]], ws[on, 0]) and torch.equal(scale[rest], sb[rest])
    assert L.ls_device_status() == 0
    now = cache.view(torch.uint8).clone()
    bad = torch.full_like(slots, -1)
    bad[0], bad[1] = R, -2
    L.ls_norm_rope(None, s["k"], s["pos"], s["inv_freq"], k_cache=cache, k_scale=scale, slots=bad)
    torch.cuda.synchronize()
    assert L.ls_device_status() == 2 and torch.equal(now, cache.view(torch.uint8))


def test_far_positions(L):
    """Positions of ten million and of 2^40: the angle is right to the last bits of its sine."""
    T, d = 6, 64
    s = make(T, 1, 1, d, 64, d, seed=4)
    pos = torch.tensor([0, 1, 10_485_759, 2 ** 31 + 7, 2 ** 40 + 1, -3], device="cuda")
    ones = torch.ones(T, 1, d, dtype=torch.bfloat16, device="cuda")
    out = L.ls_norm_rope(ones, None, pos, s["inv_freq"], fp8=False)[0].double().cpu().numpy()
    p, f = pos.double().cpu().numpy(), s["inv_freq"].double().cpu().numpy()
    a = p[:, None] * f[None, :]
    ref = np.concatenate([np.cos(a) - np.sin(a), np.cos(a) + np.sin(a)], axis=1)[:, None, :]
    # the fp64 product itself is off by 2^-53 of 2^40 turns at most: 2e-4
    assert np.all(np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + FINE + np.abs(p)[:, None, None] * 2.0 ** -51)


def test_rows_of_zeros_and_nan(L):
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    x[1, 1] = 5.0
    x[2, 0, 3] = float("nan")
    pos = torch.arange(3, device="cuda")
    f = torch.ones(32, device="cuda")
    for norm in ("none", "rms", "layer"):
        y, sc, _, _ = L.ls_norm_rope(x, None, pos, f, q_norm=norm, fp8=True)
        assert torch.all(sc[0] == 1) and torch.all(y[0].float() == 0) and sc[1, 0] == 1
        assert torch.isfinite(y[2, 1].float()).all()
        y, _, _, _ = L.ls_norm_rope(x, None, pos, f, q_norm=norm)
        assert torch.isnan(y[2, 0, 3 if norm == "none" else 100].float()) and torch.isfinite(y[:2].float()).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("off", [0, 8, 32, 5])
def test_elements_outside_the_rotation(L, off, interleaved):
    """Elements outside the rotated part keep their values, infinities and NaN among them (a NaN comes back as the
    conversion's own, 0x7fff: PTX cvt to bf16x2 keeps no payload)."""
    g = torch.Generator().manual_seed(off)
    x = torch.randn(3, 5, 128, generator=g).to(torch.bfloat16).cuda()
    x[:, :, 100], x[:, :, 110], x[:, 2, 90] = float("inf"), float("nan"), -float("inf")
    f = torch.ones(16, device="cuda")
    y = L.ls_norm_rope(x, None, torch.arange(3, device="cuda") + 1, f, rope_off=off, interleaved=interleaved)[0]
    same = ((y.view(torch.int16) == x.view(torch.int16)) | (torch.isnan(x) & torch.isnan(y))).cpu()
    assert same[:, :, :off].all() and same[:, :, off + 32:].all() and not same[:, :, off:off + 32].all()
    assert torch.isfinite(y[:, :, off:off + 32].float()).all()


def test_graph_and_stream(L):
    s = make(9, 32, 1, 128, 64, 128, seed=6)
    want = L.ls_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], q_norm="rms", k_norm="rms", fp8=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = L.ls_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], q_norm="rms", k_norm="rms", fp8=True, stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = L.ls_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], q_norm="rms", k_norm="rms", fp8=True)
    g.replay()
    torch.cuda.synchronize()
    for w, a, b in zip(want, got, cap):
        assert torch.equal(w.view(torch.uint8), a.view(torch.uint8))
        assert torch.equal(w.view(torch.uint8), b.view(torch.uint8))


def test_serving_step(L):
    """A step as a layer runs it: indexer queries and keys normed, rotated and written as fp8, the indexer's scores
    over the cache, the latent rows written, the window attended, the long-range selection attended, the parts
    joined."""
    T, N = 2, 700
    g = torch.Generator().manual_seed(8)
    rnd = lambda *sh: torch.randn(*sh, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    f = (10000.0 ** (-torch.arange(0, 64, 2).double() / 64)).float().cuda()
    k8 = torch.zeros(N, 128, device="cuda").to(torch.float8_e4m3fn)
    ks = torch.ones(N, device="cuda")
    pos = torch.arange(N, device="cuda")
    L.ls_norm_rope(None, rnd(N, 1, 128), pos, f, k_norm="layer", k_cache=k8, k_scale=ks, slots=pos)
    q8, qs, _, _ = L.ls_norm_rope(rnd(T, 32, 128), None, pos[-T:], f, fp8=True)
    w = torch.rand(1, T, 32, generator=g).cuda()
    scores = L.ls_indexer_score_fp8(q8[None], qs[None], w, k8[None], ks[None], q_pos=pos[-T:][None].contiguous(),
                                    stride=1)
    kd = k8.double().cpu() * ks.double().cpu()[:, None]
    qd = q8.double().cpu() * qs.double().cpu()[..., None]
    ref = torch.einsum("th,thn->tn", w[0].double().cpu(), torch.einsum("thd,nd->thn", qd, kd).clamp(min=0))
    seen = (pos[None, :] < pos[-T:, None] + 1).cpu()
    assert torch.equal(torch.isfinite(scores[0].cpu()), seen)
    assert ((scores[0].double().cpu() - ref)[seen].abs() <= 1e-4 * ref.max()).all()
    latent = torch.zeros(N, 576, dtype=torch.bfloat16, device="cuda")
    L.ls_norm_rope(None, rnd(N, 1, 576), pos, f, k_norm="rms", norm_dim=512, rope_off=512, interleaved=True,
                   k_cache=latent, slots=pos)
    q = L.ls_norm_rope(rnd(T, 128, 576), None, pos[-T:], f, rope_off=512, interleaved=True)[0]
    far, _ = L.ls_topk_select(scores[0, :, :500].contiguous(), 64)
    start, kv = torch.tensor([0, T], dtype=torch.int32).cuda(), torch.tensor([N], dtype=torch.int32).cuda()
    near, nl = L.ls_window_attention(q, latent, start, kv, window=100, n_sink=0, out_dtype=torch.float32)
    fo, fl = L.ls_sparse_attention(q, latent, far)
    o, z = L.ls_attention_merge(torch.stack([near, fo]), torch.stack([nl, fl]))
    for t in range(T):
        rows = far[t].tolist() + list(range(N - T + t - 99, N - T + t + 1))
        c = latent[rows].double()
        zz = q[t].double() @ c.T / 24
        assert (torch.logsumexp(zz, 1) - z[t]).abs().max() <= 1e-3
        assert (torch.softmax(zz, 1) @ c[:, :512] - o[t]).abs().max() <= (2.0 ** -8 / (1 - 2.0 ** -8) + 3e-4) * c.abs().max()
    assert L.ls_device_status() == 0


def test_refusals(L):
    s = make(4, 2, 1, 128, 64, 128, seed=7)
    a = (s["q"], s["k"], s["pos"], s["inv_freq"])
    cache = torch.zeros(9, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(4, device="cuda")
    for kw in (dict(norm_dim=100, q_norm="rms"), dict(rope_off=65), dict(rope_off=-1), dict(eps=-1.0),
               dict(eps=float("nan"))):
        with pytest.raises(L.LSError):
            L.ls_norm_rope(*a, **kw)
    for kw in (dict(q_norm="batch"), dict(q_weight=s["qw"]), dict(k_cache=cache), dict(slots=slots),
               dict(k_cache=cache, slots=slots[:3]), dict(k_cache=cache[:, :64].contiguous(), slots=slots),
               dict(k_norm="rms", k_weight=s["kw"][:64]), dict(k_cache=cache, slots=slots, fp8=True),
               dict(k_cache=cache, slots=slots, k_scale=torch.ones(9, device="cuda")),
               dict(k_cache=cache.to(torch.float8_e4m3fn), slots=slots)):
        with pytest.raises((ValueError, TypeError)):
            L.ls_norm_rope(*a, **kw)
    for bad in ((None, None), (s["q"].float(), None), (s["q"].transpose(1, 2), None), (s["q"].cpu(), None),
                (s["q"], s["k"][:2]), (s["q"][0], None)):
        with pytest.raises((ValueError, TypeError)):
            L.ls_norm_rope(*bad, s["pos"], s["inv_freq"])
    with pytest.raises(ValueError):
        L.ls_norm_rope(s["q"], None, None, s["inv_freq"])
    with pytest.raises(ValueError):
        L.ls_norm_rope(s["q"], None, s["pos"][:1], s["inv_freq"])
