"""Parity of the window and the tree attention (CUDA, through the C ABI) with the fp64 oracle.

Tolerances, from the arithmetic.  A weight enters the value contraction
rounded to bf16, w_i (1 + e_i) with |e_i| <= 2^-8 (half a step), and the
output is divided by the sum of the rounded weights.  With the weights summing
to 1 and e the weighted mean of the e_i, the error of an output is
sum w_i (e_i - e) v_i / (1 + e); sum w_i |e_i - e| is a mean deviation inside
[-2^-8, 2^-8], at most 2^-8, so it is at most 2^-8 / (1 - 2^-8) * max |v|.  A
bf16 output adds half a step, 2^-8 of itself.  A logit is accumulated over 36
steps of 16 exact products, each rounded to fp32 (at most 2^-23 of the partial
sum where the hardware truncates); the sum of the products' magnitudes times
the scale is about 23 for these inputs, so a logit is below 36 * 2^-23 * 23 =
1e-4 off, which moves a weight by 1e-4 of itself and lse by 1e-4.

Inputs of the kind "marks" make every weight an output of its own: row j has
the value 1 in column j % 512 and 0 elsewhere, so an output is a sum of
weights, and its relative error is at most 2 * 2^-8 (|e_i - e|) plus half a
bf16 step of the output where that is bf16; a missed, doubled or foreign row
shows as an error of 100 percent in its column.
"""

import numpy as np
import pytest
import torch

from oracle.attention import tree_attention, window_attention
from parity_util import dev

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -8
LOGIT = 1e-4


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_indexer_lightning_b200 import build as b
    b.build()
    import sparse_attention_indexer_lightning_b200 as lib
    return lib


def make(ns, lens, H, kind="random", seed=0, drafted=False, gap=3, pad=0):
    """Queries, latent rows (fp64 and bf16) and the batch's tables; `gap` unused rows behind each sequence and
    `pad` tokens before the first and behind the last."""
    rng = np.random.default_rng(seed)
    T = sum(ns) + 2 * pad
    caps = [m + (n if drafted else 0) + gap for n, m in zip(ns, lens)]
    off = np.concatenate([[0], np.cumsum(caps)[:-1]]).astype(np.int64)
    lat = rng.standard_normal((sum(caps) + 1, 576))
    if kind == "marks":
        for b, c in enumerate(caps):
            for j in range(c):
                lat[off[b] + j, :512] = 0.0
                lat[off[b] + j, j % 512] = 1.0
    lat = torch.from_numpy(lat).to(torch.bfloat16)
    q = torch.from_numpy(rng.standard_normal((T, H, 576)) * 1.5).to(torch.bfloat16)
    start = (pad + np.concatenate([[0], np.cumsum(ns)])).astype(np.int32)
    return dict(q=q, lat=lat, start=start, lens=np.asarray(lens, np.int32), off=off, ns=ns, H=H, T=T, rng=rng)


def check(d, out, lse, ro, rl, kind, what=""):
    bf16 = out.dtype == torch.bfloat16
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    a, b = int(d["start"][0]), int(d["start"][-1])
    out, lse, ro, rl = out[a:b], lse[a:b], ro[a:b], rl[a:b]
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty), f"{what}: empty rows"
    assert np.all(out[empty] == 0), f"{what}: empty rows must give zeros"
    assert np.all(np.abs(lse[~empty] - rl[~empty]) <= LOGIT * (1 + np.abs(rl[~empty]))), what
    if kind == "marks":
        tol = ro * (2 * STEP / (1 - STEP) + (STEP if bf16 else 0) + 3 * LOGIT) + 1e-30
    else:
        vmax = np.abs(d["lat"].double().numpy()[:, :512][np.isfinite(d["lat"].double().numpy()[:, :512])]).max()
        tol = vmax * (STEP / (1 - STEP) + 3 * LOGIT) + (STEP * np.abs(ro) * (1 + STEP) if bf16 else 0)
    err = np.abs(out - ro)
    assert np.all(err <= tol), f"{what}: {np.max(err - tol):.3e} over the bound"


def window(L, d, window, align, n_sink, kind="random", scale=None, what="", dtype=torch.bfloat16, **kw):
    scale = 576 ** -0.5 if scale is None else scale
    out, lse = L.ls_window_attention(d["q"].cuda(), d["lat"].cuda(), dev(d["start"]), dev(d["lens"]),
                                     row_off=dev(d["off"]), window=window, align=align, n_sink=n_sink, scale=scale,
                                     out_dtype=dtype, **kw)
    torch.cuda.synchronize()
    assert L.ls_device_status() == 0
    ro, rl = window_attention(d["q"].double().numpy(), d["lat"].double().numpy(), d["start"], d["lens"], d["off"],
                              window, align, n_sink, scale)
    check(d, out, lse, ro, rl, kind, what)
    return out, lse


WINDOWS = [
    # tokens, rows, heads, window, align, sinks
    ([1], [1], 128, 512, 1, 4),
    ([1], [0], 16, 512, 1, 4),                       # position -1: nothing to see
    ([3], [2], 5, 4, 1, 1),                          # the first token sees nothing
    ([1], [700], 128, 512, 1, 4),
    ([1, 1, 1, 1], [5, 64, 517, 900], 128, 512, 1, 4),
    ([1] * 9, [1, 2, 16, 17, 63, 64, 65, 128, 129], 16, 64, 1, 0),
    ([7], [300], 24, 1, 1, 0),                       # each token sees itself
    ([7], [300], 24, 1, 1, 5),
    ([40], [1200], 16, 100, 1, 70),                  # sinks longer than a tile
    ([40], [130], 16, 100, 1, 70),                   # sinks and window meet
    ([33, 0, 2, 65], [33, 50, 400, 66], 3, 17, 1, 4),
    ([5, 70], [600, 1100], 16, 1, 512, 4),           # the block window
    ([9], [40], 130, 13, 7, 2),
    ([3], [2000], 256, 1500, 1, 4),
    ([6], [6], 1, 1 << 20, 1, 0),
    ([200], [300], 1, 30, 1, 4),
    ([4], [90], 1024, 64, 1, 1),
]


@pytest.mark.parametrize("kind", ["random", "marks"])
@pytest.mark.parametrize("case", WINDOWS, ids=[str(i) for i in range(len(WINDOWS))])
def test_window(L, case, kind):
    ns, lens, H, w, align, sinks = case
    d = make(ns, lens, H, kind, seed=len(ns) * 100 + H)
    window(L, d, w, align, sinks, kind)
    window(L, d, w, align, sinks, kind, dtype=torch.float32)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_window_scales(L, scale):
    """scale 0 weighs all visible rows alike; a large one lets a row's maximum grow from tile to tile."""
    d = make([3], [700], 16, "marks", seed=5)
    if scale == 1.0:
        # logits rise along the window, so every tile raises the maximum by more than a rescale's threshold
        lat = d["lat"].double().numpy()
        lat[:, 512:] = 0.0
        lat[:, 512] = np.arange(lat.shape[0]) // 16
        d["lat"] = torch.from_numpy(lat).to(torch.bfloat16)
        q = np.zeros(d["q"].shape)
        q[:, :, 512] = 1.0
        q[:, 3, 512] = -1.0
        d["q"] = torch.from_numpy(q).to(torch.bfloat16)
    window(L, d, 512, 1, 4, "marks", scale=scale)


def tree_bits(branches, words):
    out = np.zeros((len(branches), words), np.uint64)
    for t, seen in enumerate(branches):
        for i in seen:
            out[t, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return out.view(np.int64)


def random_tree(rng, ns, pad=0):
    branches = [set() for _ in range(pad)]
    for n in ns:
        mine = []
        for i in range(n):
            parent = int(rng.integers(-1, i)) if i else -1
            mine.append((set(mine[parent]) if parent >= 0 else set()) | {i})
        branches += mine
    return branches + [set() for _ in range(pad)]


def tree(L, d, branches, kind="random", window=0, align=1, n_sink=0, what="", dtype=torch.bfloat16, words=None, **kw):
    words = (max(d["ns"]) + 63) // 64 if words is None else words
    out, lse = L.ls_tree_attention(d["q"].cuda(), d["lat"].cuda(), dev(d["start"]), dev(d["lens"]),
                                   dev(tree_bits(branches, words)), row_off=dev(d["off"]), window=window,
                                   align=align, n_sink=n_sink, out_dtype=dtype, **kw)
    torch.cuda.synchronize()
    assert L.ls_device_status() == 0
    ro, rl = tree_attention(d["q"].double().numpy(), d["lat"].double().numpy(), d["start"], d["lens"], d["off"],
                            branches, window, align, n_sink, 576 ** -0.5)
    check(d, out, lse, ro, rl, kind, what)
    return out, lse


def tree_call(L, d, branches, **kw):
    words = (max(d["ns"]) + 63) // 64
    return L.ls_tree_attention(d["q"].cuda(), d["lat"].cuda(), dev(d["start"]), dev(d["lens"]),
                               dev(tree_bits(branches, words)), row_off=dev(d["off"]), **kw)


TREES = [
    # tokens, context, heads, window, align, sinks
    ([1], [0], 128, 0, 1, 0),
    ([5], [100], 128, 0, 1, 0),
    ([1], [3000], 128, 0, 1, 0),
    ([64], [64], 16, 0, 1, 0),
    ([65], [63], 8, 0, 1, 0),
    ([130], [40], 3, 0, 1, 0),
    ([8, 3, 0, 17], [1000, 0, 30, 129], 16, 0, 1, 0),
    ([2], [5000], 16, 0, 1, 0),
    ([20], [900], 16, 128, 1, 4),
    ([20], [900], 16, 10, 1, 0),
    ([9, 4], [700, 520], 130, 1, 512, 4),
]


@pytest.mark.parametrize("kind", ["random", "marks"])
@pytest.mark.parametrize("case", TREES, ids=[str(i) for i in range(len(TREES))])
def test_tree(L, case, kind):
    ns, lens, H, w, align, sinks = case
    d = make(ns, lens, H, kind, seed=len(ns) * 100 + H + 1, drafted=True)
    branches = random_tree(d["rng"], ns)
    tree(L, d, branches, kind, w, align, sinks)
    tree(L, d, branches, kind, w, align, sinks, dtype=torch.float32, max_ctx=max(lens))


def test_tree_masks_that_leave_nothing(L):
    """No context and no bit: zeros and -inf; bits at or past the sequence's tokens are not seen; more words than
    needed; a token that does not see itself."""
    d = make([6, 4], [0, 70], 16, "marks", seed=9, drafted=True)
    branches = [set(), {0}, {0, 1, 5}, set(), {5}, {4}] + [set(), {0, 3}, {1}, {63, 100}]
    out, lse = tree(L, d, branches, "marks", words=2)
    assert torch.all(out[0] == 0) and torch.all(torch.isinf(lse[0]))


def _same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_masked_rows_may_hold_anything(L):
    """NaN and infinities in rows that nobody sees, behind the last row of a sequence, and in rows of a sibling
    branch leave the other outputs as they are, bit for bit; the tokens that see such a row are NaN."""
    d = make([3, 20], [1500, 45], 16, seed=3)
    out, lse = window(L, d, 200, 1, 4)
    lat = d["lat"].clone()
    seen = set()
    for b, (n, m) in enumerate(zip(d["ns"], d["lens"])):
        for p in range(m - n, m):
            seen |= {int(d["off"][b]) + j for j in range(p + 1) if j < 4 or j > p - 200}
    hidden = [r for r in range(lat.shape[0]) if r not in seen]
    for i, r in enumerate(hidden):
        lat[r] = (float("nan"), float("inf"), -float("inf"))[i % 3]
    d2 = dict(d, lat=lat)
    args = (dev(d["start"]), dev(d["lens"]))
    out2, lse2 = L.ls_window_attention(d["q"].cuda(), lat.cuda(), *args, row_off=dev(d["off"]), window=200, n_sink=4)
    assert _same(out, out2) and _same(lse, lse2)

    # a window's first row, seen by the earlier tokens of the tile only
    lat = d["lat"].clone()
    lat[1500 - 3 - 200 + 1, 17] = float("inf")            # first row of token 0's window
    out2, lse2 = L.ls_window_attention(d["q"].cuda(), lat.cuda(), *args, row_off=dev(d["off"]), window=200, n_sink=4)
    assert _same(out[1:], out2[1:]) and _same(lse[1:], lse2[1:])

    # two branches: {0, 2} and {1, 3}; row 0 of the drafted ones is not finite
    d = make([4], [70], 16, seed=4, drafted=True)
    branches = [{0}, {1}, {0, 2}, {1, 3}]
    out, lse = tree(L, d, branches)
    for bad in (float("nan"), float("inf")):
        lat = d["lat"].clone()
        lat[70, 100:140] = bad
        out2, lse2 = L.ls_tree_attention(d["q"].cuda(), lat.cuda(), dev(d["start"]), dev(d["lens"]),
                                         dev(tree_bits(branches, 1)), row_off=dev(d["off"]))
        assert _same(out[[1, 3]], out2[[1, 3]]) and _same(lse[[1, 3]], lse2[[1, 3]])
        if bad != bad:
            assert torch.isnan(out2[[0, 2]].float()).all() and torch.isnan(lse2[[0, 2]]).all()
    # a query that is NaN spoils its own row only
    q = d["q"].clone()
    q[2, 5, 7] = float("nan")
    out2, lse2 = L.ls_tree_attention(q.cuda(), d["lat"].cuda(), dev(d["start"]), dev(d["lens"]),
                                     dev(tree_bits(branches, 1)), row_off=dev(d["off"]))
    keep = torch.ones(4, 16, dtype=torch.bool)
    keep[2, 5] = False
    assert _same(out[keep.cuda()], out2[keep.cuda()]) and torch.isnan(out2[2, 5].float()).all()


def test_rows_outside_the_sequences_are_left(L):
    d = make([2, 5], [80, 700], 16, seed=6, pad=3)
    for kw in (dict(window=64, n_sink=4), dict(window=5000, n_sink=0)):
        out = torch.full((d["T"], 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        window(L, d, kw["window"], 1, kw["n_sink"], out=out)
        assert torch.all(out[:3] == 7) and torch.all(out[-3:] == 7)


def test_outputs_given_and_left(L):
    """Cut work (one item over many pairs) and whole items: tokens outside the sequences keep what out held, lse is
    optional, and max_q bounds what is computed."""
    for lens, H in (([9000], 16), ([30], 128)):
        d = make([3], lens, H, "marks", seed=21, drafted=True, pad=2)
        branches = random_tree(d["rng"], d["ns"], pad=2)
        want, _ = tree(L, d, branches, "marks")
        out = torch.full((d["T"], H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        got, none = tree_call(L, d, branches, out=out, want_lse=False, max_q=3)
        assert none is None and got is out and _same(got[2:5], want[2:5])
        assert torch.all(out[:2] == 7) and torch.all(out[5:] == 7)
    d = make([3], [700], 128, "marks", seed=22, pad=1)
    out = torch.full((d["T"], 128, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    args = (d["q"].cuda(), d["lat"].cuda(), dev(d["start"]), dev(d["lens"]))
    want, _ = L.ls_window_attention(*args, row_off=dev(d["off"]), window=600)
    L.ls_window_attention(*args, row_off=dev(d["off"]), window=600, out=out, want_lse=False, max_q=3)
    assert _same(out[1:4], want[1:4]) and torch.all(out[0] == 7) and torch.all(out[4] == 7)
    assert L.ls_device_status() == 0


def test_fewer_mask_words_than_drafted_rows(L):
    """Drafted rows past the mask's words are not seen, and no word past a token's own is read (the last token's mask
    ends with the tensor)."""
    d = make([150], [90], 16, "marks", seed=24, drafted=True)
    branches = [{i for i in range(150) if i % 3 == t % 3 and i <= t} for t in range(150)]
    cut = [{i for i in b if i < 64} for b in branches]
    tree(L, d, cut, "marks", words=1)
    d = make([8] * 12, [100] * 12, 16, "marks", seed=25, drafted=True)   # one word does for all, whatever T is
    tree(L, d, random_tree(d["rng"], d["ns"]), "marks", words=1)


def test_two_calls_at_once(L):
    """Two calls on two streams, each with its workspace, beside one another, and sequences that share their rows."""
    d = make([2, 2], [5000, 5000], 16, seed=23, drafted=True)
    d["off"][1] = d["off"][0]                             # the second sequence reads the first one's rows
    branches = [{0}, {0, 1}] * 2
    want = tree(L, d, branches)
    args = (d["q"].cuda(), d["lat"].cuda(), dev(d["start"]), dev(d["lens"]), dev(tree_bits(branches, 1)))
    off = dev(d["off"])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for i in range(20):
        outs.append(L.ls_tree_attention(*args, row_off=off, stream=streams[i % 2]))
    torch.cuda.synchronize()
    for o, z in outs:
        assert _same(o, want[0]) and _same(z, want[1])


def test_splits_agree_and_repeat(L):
    """How the work is split does not change what is computed beyond fp32 rounding of the joined parts; the same call
    gives the same bits."""
    d = make([3], [6000], 16, seed=8, drafted=True)
    branches = random_tree(d["rng"], d["ns"])
    runs = [tree(L, d, branches, dtype=torch.float32, max_ctx=m) for m in (0, 64, 6000)]
    again = tree(L, d, branches, dtype=torch.float32, max_ctx=6000)
    assert _same(runs[2][0], again[0]) and _same(runs[2][1], again[1])
    for o, z in runs:
        # each part rounds its weights against its own reference, so parts agree to the weights' rounding
        assert (o - runs[0][0]).abs().max() <= 2 * STEP * d["lat"].abs().max()
        assert (z - runs[0][1]).abs().max() <= LOGIT


@pytest.mark.parametrize("case", [WINDOWS[i] for i in (7, 9, 12, 15, 16)], ids=["7", "9", "12", "15", "16"])
def test_every_call_gives_the_same_bits(L, case):
    """300 calls, bit for bit: what one warp reads of another's maxima, sums and items has been written by then."""
    ns, lens, H, w, align, sinks = case
    d = make(ns, lens, H, seed=H)
    args = (d["q"].cuda(), d["lat"].cuda(), dev(d["start"]), dev(d["lens"]))
    kw = dict(row_off=dev(d["off"]), window=w, align=align, n_sink=sinks, out_dtype=torch.float32)
    out, lse = L.ls_window_attention(*args, **kw)
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        o, z = L.ls_window_attention(*args, **kw)
        bad += (o.view(torch.int32) != out.view(torch.int32)).sum() + (z.view(torch.int32) != lse.view(torch.int32)).sum()
    assert int(bad) == 0


def test_ragged_trees_cut_into_equal_runs(L):
    """More items than pairs, of very different lengths: cuts go through many items, some items lie in one run and
    some runs inside one item; one item's parts over all pairs; a sequence without tokens, one without rows."""
    for ns, lens, H in (([9, 0, 1, 30, 2, 17], [2000, 50, 0, 300, 5000, 130], 128), ([1], [20000], 128),
                        ([3, 3], [0, 9000], 24), ([100], [700], 128)):
        d = make(ns, lens, H, "marks", seed=len(ns) + H, drafted=True)
        branches = random_tree(d["rng"], ns)
        tree(L, d, branches, "marks", dtype=torch.float32, max_ctx=max(lens))
        tree(L, d, branches, "marks")


def test_far_rows(L):
    """Rows more than 2^31 elements and 2^32 bytes into the cache."""
    R = 4_200_000
    d = make([2], [150], 16, "marks", seed=10)
    lat = torch.zeros(R, 576, dtype=torch.bfloat16, device="cuda")
    lat[R - 160:R - 10] = d["lat"][:150].cuda()
    off = torch.tensor([R - 160], device="cuda")
    out, lse = L.ls_window_attention(d["q"].cuda(), lat, dev(d["start"]), dev(d["lens"]), row_off=off, window=100)
    ro, rl = window_attention(d["q"].double().numpy(), d["lat"].double().numpy(), d["start"], d["lens"], [0], 100, 1,
                              4, 576 ** -0.5)
    check(d, out, lse, ro, rl, "marks")
    assert L.ls_device_status() == 0


def test_bad_tables_set_the_fault(L):
    d = make([3, 2], [90, 50], 16, seed=11)
    q, lat = d["q"].cuda(), d["lat"].cuda()
    good = window(L, d, 64, 1, 4)

    def call(start=d["start"], lens=d["lens"], off=d["off"], **kw):
        r = L.ls_window_attention(q, lat, dev(np.asarray(start, np.int32)), dev(np.asarray(lens, np.int32)),
                                  row_off=dev(np.asarray(off, np.int64)), window=64, **kw)
        torch.cuda.synchronize()
        return r, L.ls_device_status()

    assert call()[1] == 0
    bad = [dict(start=[0, 4, 3]), dict(start=[0, 3, 6]), dict(start=[-1, 3, 5]), dict(lens=[90, 1000]),
           dict(lens=[-1, 50]), dict(lens=[90, 2 ** 31 - 1]), dict(off=[0, -5]), dict(off=[0, 10 ** 12])]
    for kw in bad:
        assert call(**kw)[1] == 2, kw
    big = make([20], [90], 16, seed=12)
    L.ls_window_attention(big["q"].cuda(), big["lat"].cuda(), dev(big["start"]), dev(big["lens"]), max_q=4)
    torch.cuda.synchronize()
    assert L.ls_device_status() == 2                      # more tokens than max_q covers
    # the other sequence of a batch with a bad row offset is computed as before
    (out, lse), st = call(off=[0, 10 ** 12])
    assert st == 2 and _same(out[:3], good[0][:3]) and torch.all(out[3:] == 0)


def test_graph_stream_and_reused_workspace(L):
    """A captured call replays on new contents of its tensors; a call on a side stream; a workspace of the caller's."""
    d = make([2], [4000], 16, seed=13, drafted=True)
    e = make([2], [4000], 16, seed=14, drafted=True)
    branches = [{0}, {0, 1}]
    want_d, want_e = tree(L, d, branches), tree(L, e, branches)
    q, lat = d["q"].cuda(), d["lat"].cuda()
    start, lens, off, mask = dev(d["start"]), dev(d["lens"]), dev(d["off"]), dev(tree_bits(branches, 1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = L.ls_tree_attention(q, lat, start, lens, mask, row_off=off, stream=side)
    side.synchronize()
    assert _same(out, want_d[0]) and _same(lse, want_d[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = L.ls_tree_attention(q, lat, start, lens, mask, row_off=off)
    g.replay()
    torch.cuda.synchronize()
    assert _same(out, want_d[0])
    q.copy_(e["q"])
    lat.copy_(e["lat"])
    g.replay()
    torch.cuda.synchronize()
    assert _same(out, want_e[0]) and _same(lse, want_e[1])
    need = L.lib().ls_tree_attention_workspace_size(1, 2, 16, 2, lat.shape[0], 0, 0, 1, 0)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out, lse = L.ls_tree_attention(q, lat, start, lens, mask, row_off=off, ws=ws)
    assert _same(out, want_e[0])
    with pytest.raises(L.LSError):
        L.ls_tree_attention(q, lat, start, lens, mask, row_off=off, ws=ws[:need - 256])
    assert L.ls_device_status() == 0


def test_joins_the_sparse_attention(L):
    """The bucket search's read list (sinks, block window, long-range keys) as one sparse attention, and as the block
    window and the sparse attention over the long-range keys, joined."""
    T, H, N = 3, 128, 2000
    d = make([T], [N], H, seed=15)
    q, lat = d["q"].cuda(), d["lat"].cuda()
    rng = np.random.default_rng(15)
    idx = np.full((T, 512), -1, np.int32)
    far = np.full((T, 100), -1, np.int32)
    for i in range(T):
        p = N - T + i
        lo = p // 128 * 128
        pick = rng.choice(np.arange(4, lo), 90, replace=False)
        far[i, :90] = pick
        all_ = list(range(4)) + list(range(lo, p + 1)) + list(pick)
        idx[i, :len(all_)] = all_
    whole, wl = L.ls_sparse_attention(q, lat, dev(idx), cuda_cores=True)
    near, nl = L.ls_window_attention(q, lat, dev(d["start"]), dev(d["lens"]), window=1, align=128, n_sink=4,
                                     out_dtype=torch.float32)
    fo, fl = L.ls_sparse_attention(q, lat, dev(far), cuda_cores=True)
    o, z = L.ls_attention_merge(torch.stack([near, fo]), torch.stack([nl, fl]))
    assert (z - wl).abs().max() <= 2 * LOGIT
    assert (o - whole).abs().max() <= (STEP / (1 - STEP) + 5 * LOGIT) * lat.abs().max()


def test_refusals(L):
    d = make([2], [50], 16, seed=16)
    q, lat, start, lens = d["q"].cuda(), d["lat"].cuda(), dev(d["start"]), dev(d["lens"])
    for kw, err in ((dict(window=0), L.LSError), (dict(align=0), L.LSError), (dict(n_sink=-1), L.LSError),
                    (dict(scale=float("nan")), L.LSError), (dict(out_dtype=torch.float16), TypeError),
                    (dict(row_off=torch.zeros(2, dtype=torch.int64, device="cuda")), ValueError)):
        with pytest.raises(err):
            L.ls_window_attention(q, lat, start, lens, **kw)
    for bad in ((q.float(), lat, start, lens), (q, lat.float(), start, lens), (q, lat, start.long(), lens),
                (q.cpu(), lat, start, lens), (q, lat, start, lens.long()), (q, lat[:, :512].contiguous(), start, lens),
                (q.transpose(0, 1), lat, start, lens), (q, lat, start[:1], lens), (q, lat.cpu(), start, lens)):
        with pytest.raises((TypeError, ValueError)):
            L.ls_window_attention(*bad)
    mask = torch.zeros(2, 1, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        L.ls_tree_attention(q, lat, start, lens, mask[:1])
    with pytest.raises(TypeError):
        L.ls_tree_attention(q, lat, start, lens, mask.int())
    with pytest.raises(L.LSError):
        L.ls_tree_attention(q, lat, start, lens, mask[:, :0].contiguous())
    # nothing to do: no tokens, no sequences
    out, lse = L.ls_window_attention(q[:0], lat, torch.zeros(1, dtype=torch.int32, device="cuda"), lens[:0])
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16)
