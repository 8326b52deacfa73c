"""The span attentions at their edges (CUDA, through the C ABI), against the fp64 oracle: maxima that grow from tile to
tile, sinks of several tiles, n_sink at the largest int, pairs that run through many items, batches whose max_q is
left at its default, more tokens than max_q, logits that are not finite, the read lists of the LSA search.
Tolerances as in test_gpu_span_attention.py.
"""

import numpy as np
import pytest
import torch

from parity_util import dev, dev_bf16
from test_gpu_span_attention import (  # noqa: F401
    L, LOGIT, STEP, _same, check, make, random_tree, tree, tree_bits, tree_call, window,
)
from workloads.synth import make_lsa

pytestmark = pytest.mark.gpu

FACTORS = (1.0, 0.75, 0.5, -1.0, 0.0, -0.25, 2.0)


def levels(d, level):
    """Logits that follow `level` (one number per latent row) times a factor of the head, in nats: column 512 holds the
    level and the query 24 times the factor (the scale is 1 / 24); values and the other logits as they were."""
    lat = d["lat"].double()
    lat[:, 512:] = 0.0
    lat[:level.shape[0], 512] = torch.from_numpy(level)
    d["lat"] = lat.to(torch.bfloat16)
    assert torch.equal(d["lat"][:level.shape[0], 512].double(), torch.from_numpy(level)), "levels that bf16 rounds"
    q = d["q"].double()
    q[:, :, 512:] = 0.0
    q[:, :, 512] = 24.0 * torch.tensor([FACTORS[h % len(FACTORS)] for h in range(d["H"])])
    d["q"] = q.to(torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ctx,drafted", [(450, 3), (512, 3), (385, 40), (640, 1), (130, 3)])
def test_maxima_that_grow_from_tile_to_tile(L, ctx, drafted, dtype):  # noqa: F811
    """16 nats a tile (23 in log2: above the 16 that force a rescale), 12 (17), 8 (11.5: every second tile), falling, flat,
    and 32: the output is rescaled in full tiles, in a tile of few rows and in the tile of the drafted rows.  max_ctx = 1
    keeps the item whole (the hint decides the split only)."""
    d = make([drafted], [ctx], 16, "marks", seed=ctx, drafted=True)
    levels(d, 16.0 * (np.arange(ctx + drafted) // 128 + (np.arange(ctx + drafted) >= ctx)))
    branches = random_tree(d["rng"], d["ns"])
    rows = d["lat"].shape[0]
    assert L.lib().ls_tree_attention_workspace_size(1, drafted, 16, drafted, rows, 1, 0, 1, 0) == 0
    tree(L, d, branches, "marks", dtype=dtype, max_ctx=1)
    tree(L, d, branches, "marks", dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_maxima_that_grow_in_whole_windows(L, dtype):  # noqa: F811
    """As many query tiles as pairs, so that each pair has one whole item: window tiles that grow, then sinks above all of
    them (the sinks come last)."""
    d = make([74], [700], 128, "marks", seed=31)
    level = 16.0 * (np.arange(700) // 128)
    level[:4] = 128.0
    levels(d, level)
    assert L.lib().ls_window_attention_workspace_size(1, 74, 128, 74, 500, 1, 4) == 0
    window(L, d, 500, 1, 4, "marks", dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_maxima_that_grow_inside_cut_runs(L, dtype):  # noqa: F811
    """One item over all pairs, four tiles a run, levels that rise over five tiles and start again."""
    ctx = 74 * 4 * 128 + 50
    d = make([1], [ctx], 16, "marks", seed=32, drafted=True)
    levels(d, 16.0 * (np.arange(ctx + 1) // 128 % 5))
    need = L.lib().ls_tree_attention_workspace_size(1, 1, 16, 1, d["lat"].shape[0], ctx, 0, 1, 0)
    assert need > 2 * 74 * 128 * 512 * 4                  # all 74 pairs
    tree(L, d, [{0}], "marks", dtype=dtype, max_ctx=ctx)


@pytest.mark.parametrize("sinks", [128, 200, 256, 300])
def test_sinks_of_several_tiles(L, sinks):  # noqa: F811
    d = make([40], [1200], 16, "marks", seed=sinks)
    window(L, d, 100, 1, sinks, "marks")
    d = make([74], [1200], 128, "random", seed=sinks)     # whole items
    window(L, d, 100, 1, sinks, "random", dtype=torch.float32)
    d = make([20], [900], 16, "marks", seed=sinks, drafted=True)
    tree(L, d, random_tree(d["rng"], [20]), "marks", window=128, n_sink=sinks)


def test_all_sinks(L):  # noqa: F811
    """n_sink at the largest int: every row is one."""
    d = make([3], [300], 16, "marks", seed=33)
    window(L, d, 1, 1, (1 << 31) - 1, "marks")


@pytest.mark.parametrize("n,H", [(500, 128), (1500, 40)])
def test_pairs_that_run_through_many_items(L, n, H):  # noqa: F811
    """Six or seven whole items a pair, so that the places of the items in shared memory come round."""
    d = make([n], [n + 20], H, "random", seed=n)
    assert L.lib().ls_window_attention_workspace_size(1, n, H, n, 20, 1, 4) == 0
    window(L, d, 20, 1, 4)


def best_us(call, n=20, tries=4):
    call()
    best = 1e30
    for _ in range(tries):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        for _ in range(n):
            call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / n)
    return best


def test_decode_batches_without_max_q(L):  # noqa: F811
    """148 single tokens: with max_q left out every pair has its two items, as with max_q = 1 (dealt by places of padded
    sequences all 148 would fall to one pair).  The two calls do the same work, so 1.5 times is far from their noise."""
    B = 148
    lens = [int(x) for x in np.random.default_rng(34).integers(1, 900, B)]
    d = make([1] * B, lens, 128, "random", seed=34)
    window(L, d, 512, 1, 4)
    window(L, d, 512, 1, 4, dtype=torch.float32, max_q=1)
    args = (d["q"].cuda(), d["lat"].cuda(), dev(d["start"]), dev(d["lens"]))
    call = lambda **kw: L.ls_window_attention(*args, row_off=dev_off, window=512, n_sink=4, **kw)  # noqa: E731
    dev_off = dev(d["off"])
    assert _same(call()[0], call(max_q=1)[0])
    assert best_us(call) < 1.5 * best_us(lambda: call(max_q=1))


@pytest.mark.parametrize("ns,H", [([0] * 70 + [1] + [0] * 40 + [3, 0, 0, 9] + [0] * 100 + [2], 128),
                                  ([1, 0] * 90, 16), ([5] * 33, 130), ([0] * 65, 16), ([90, 1, 0, 2], 128)])
def test_ragged_batches_without_max_q(L, ns, H):  # noqa: F811
    """Sequences without tokens before, between and behind the others, more of them than are looked at together; whole
    items and cut ones."""
    lens = [int(x) for x in np.random.default_rng(len(ns)).integers(0, 300, len(ns))]
    d = make(ns, lens, H, "marks", seed=len(ns), drafted=True)
    branches = random_tree(d["rng"], ns)
    if sum(ns):
        tree(L, d, branches, "marks")                     # contexts as long as the cache, as far as the host knows: cut
        tree(L, d, branches, "marks", max_ctx=1)          # whole
        d = make(ns, [n + m for n, m in zip(ns, lens)], H, "marks", seed=len(ns))
        window(L, d, 64, 1, 4, "marks")
    else:
        d = make(ns, lens, H, "marks", seed=len(ns), drafted=True, pad=2)
        out = torch.full((4, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        L.ls_tree_attention(d["q"].cuda(), d["lat"].cuda(), dev(d["start"]), dev(d["lens"]),
                            torch.zeros(4, 1, dtype=torch.int64, device="cuda"), row_off=dev(d["off"]), out=out)
        assert torch.all(out == 7) and L.ls_device_status() == 0


def test_more_tokens_than_max_q(L):  # noqa: F811
    """A sequence with more tokens than max_q sets the fault, whatever room the last tile of query rows has left; max_q = 0
    is right for a batch without tokens, and no other."""
    d = make([3, 5], [40, 50], 16, "marks", seed=35, pad=1)
    args = (d["q"].cuda(), d["lat"].cuda(), dev(d["start"]), dev(d["lens"]))

    def status(call, *a, **kw):
        r = call(*a, row_off=dev(d["off"]), **kw)
        torch.cuda.synchronize()
        return r, L.ls_device_status()

    assert status(L.ls_window_attention, *args, max_q=5)[1] == 0
    mask = torch.zeros(10, 1, dtype=torch.int64, device="cuda")
    for m in (4, 3, 1, 0):
        assert status(L.ls_window_attention, *args, max_q=m)[1] == 2, m
        assert status(L.ls_tree_attention, *args[:3], dev(np.array([20, 20], np.int32)), mask, max_q=m)[1] == 2, m
        long = dev(np.array([20, 20], np.int32))
        assert status(L.ls_tree_attention, *args[:3], long, mask, max_q=m, max_ctx=1)[1] == 2, m
    out = torch.full((10, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    none = (args[0], args[1], torch.full((3,), 4, dtype=torch.int32, device="cuda"), args[3])
    assert status(L.ls_window_attention, *none, max_q=0, out=out)[1] == 0 and torch.all(out == 7)


# Visible rows that are not finite: a context of 300 rows, so that the bad row lies in a tile that every token
# sees whole (5, 130) or in one with places behind the last row (290).
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("max_ctx", [1, 0])
@pytest.mark.parametrize("bad_row", [5, 130, 290])
def test_visible_infinities(L, bad_row, max_ctx, dtype):  # noqa: F811
    """A visible row with an infinity or a NaN in a value column: the (token, head) row is NaN where its logit is NaN or
    +inf; where it is -inf (a weight of 0) that column is, and lse stays; in a whole tile and in one with masks alike.
    An infinity in a key-only element with a logit of -inf weighs 0."""
    d = make([2], [300], 16, seed=36, drafted=True)
    branches = [{0}, {0, 1}]
    q = d["q"].double()
    q[:, :, 17] = torch.tensor([1.0, -1.0] * 8)
    q[:, :, 550] = torch.tensor([-1.0] * 12 + [1.0] * 4)
    d["q"] = q.to(torch.bfloat16)
    for value, odd in ((float("inf"), 0), (-float("inf"), 1), (float("nan"), None)):
        lat = d["lat"].clone()
        lat[bad_row, 17] = value
        out, lse = tree_call(L, dict(d, lat=lat), branches, out_dtype=dtype, max_ctx=max_ctx)
        nan = slice(None) if odd is None else slice(odd, None, 2)
        assert torch.isnan(out[:, nan].float()).all() and torch.isnan(lse[:, nan]).all()
        assert torch.isnan(out[:, :, 17].float()).all()
        if odd is not None:                               # the same lse as without that row
            low = slice(1 - odd, None, 2)
            assert not torch.isnan(lse[:, low]).any()
            without = lat.clone()
            without[bad_row] = 0.0
            without[bad_row, 17] = 2.0 ** 100 if odd == 0 else -2.0 ** 100
            assert _same(lse[:, low].contiguous(),
                         tree_call(L, dict(d, lat=without), branches, max_ctx=max_ctx)[1][:, low].contiguous())
    lat = d["lat"].clone()
    lat[bad_row, 550] = float("inf")
    e = dict(d, lat=d["lat"].clone())
    out, lse = tree_call(L, dict(d, lat=lat), branches, out_dtype=dtype, max_ctx=max_ctx)
    assert torch.isnan(out[:, 12:].float()).all() and torch.isnan(lse[:, 12:]).all()
    # heads 0 .. 11: the same as without that row, which a level of -2^100 in a key-only element takes away
    e["lat"][bad_row, 550] = 2.0 ** 100
    want, wl = tree_call(L, e, branches, out_dtype=dtype, max_ctx=max_ctx)
    assert _same(out[:, :12].contiguous(), want[:, :12].contiguous())
    assert _same(lse[:, :12].contiguous(), wl[:, :12].contiguous())
    assert L.ls_device_status() == 0


def test_infinities_that_a_neighbour_does_not_see(L):  # noqa: F811
    """The first row of a window, seen by the tile's first token alone, with a logit of -inf: the column that is infinite
    there is NaN in that token's rows and its lse is as without that row; the others are as they were; and so it is when
    the token is alone in its batch."""
    d = make([3], [700], 16, seed=37)
    q = d["q"].double()
    q[:, :, 17] = -1.0
    d["q"] = q.to(torch.bfloat16)
    first = 700 - 3 - 200 + 1
    lat = d["lat"].clone()
    lat[first, 17] = float("inf")
    good, gl = window(L, d, 200, 1, 4)
    args = (dev(d["start"]), dev(d["lens"]))
    out, lse = L.ls_window_attention(d["q"].cuda(), lat.cuda(), *args, row_off=dev(d["off"]), window=200, n_sink=4)
    assert _same(out[1:], good[1:]) and _same(lse[1:], gl[1:])
    assert torch.isnan(out[0, :, 17].float()).all() and torch.isfinite(lse).all()
    one = dev(np.array([0, 1], np.int32))
    out, alone = L.ls_window_attention(d["q"][:1].cuda(), lat.cuda(), one, dev(np.array([698], np.int32)), window=200,
                                       n_sink=4)
    assert torch.isnan(out[0, :, 17].float()).all() and (alone[0] - lse[0]).abs().max() <= 2 * LOGIT


@pytest.mark.parametrize("max_ctx", [1, 0])
def test_logits_below_the_fp32_range(L, max_ctx):  # noqa: F811
    """A logit that leaves fp32 downwards (finite elements) weighs 0, in a whole tile and in one with masks."""
    d = make([2], [300], 16, "marks", seed=38, drafted=True)
    lat, q = d["lat"].double(), d["q"].double()
    lat[:, 560], q[:, :, 560] = 0.0, -2.0 ** 90
    for r in (7, 140, 295):
        lat[r, 560] = 2.0 ** 60
    d["lat"], d["q"] = lat.to(torch.bfloat16), q.to(torch.bfloat16)
    tree(L, d, [{0}, {1}], "marks", dtype=torch.float32, max_ctx=max_ctx)


@pytest.mark.parametrize("H", [16, 128])
def test_read_lists_of_the_lsa_search(L, H):  # noqa: F811
    """keys_out holds the sinks and the window in front of the long-range keys: the sparse attention over the whole list,
    and the block window joined with the sparse attention over the list without its sinks and window, agree; the two
    whole parts joined would count sinks and window twice."""
    T, N, block, n_sink = 24, 2100, 512, 4
    s = make_lsa(T, N, block_keys=block, seed=39, chunk=True)
    pos = dev(s["q_pos"])
    assert s["q_pos"].tolist() == list(range(N - T, N))
    keys, n = L.ls_lsa_flat_select(dev_bf16(s["q_idx"]), pos, dev_bf16(s["centroids"]), dev(s["bucket_off"]),
                                   dev(s["bucket_mem"]), block_keys=block, n_sink=n_sink, top_p=64, budget=200)
    d = make([T], [N], H, seed=39)
    q, lat = d["q"].cuda(), d["lat"].cuda()
    whole, wl = L.ls_sparse_attention(q, lat, keys, cuda_cores=True)
    lo = (pos // block * block)[:, None]
    far = torch.where((keys < n_sink) | (keys >= lo), torch.full_like(keys, -1), keys)
    assert torch.equal((far >= 0).sum(1), n - n_sink - (pos - lo[:, 0] + 1)) and int((far >= 0).sum()) == 200 * T
    near, nl = L.ls_window_attention(q, lat, dev(d["start"]), dev(d["lens"]), window=1, align=block, n_sink=n_sink,
                                     out_dtype=torch.float32)
    fo, fl = L.ls_sparse_attention(q, lat, far, cuda_cores=True)
    o, z = L.ls_attention_merge(torch.stack([near, fo]), torch.stack([nl, fl]))
    assert (z - wl).abs().max() <= 2 * LOGIT
    assert (o - whole).abs().max() <= (STEP / (1 - STEP) + 5 * LOGIT) * lat.abs().max()
    assert L.ls_device_status() == 0


@pytest.mark.parametrize("whole", [True, False])
def test_masked_rows_that_are_not_finite_every_time(L, whole):  # noqa: F811
    """300 calls bit for bit those over clean rows, with NaN and infinities in every masked row, many tiles a pair and
    staged values to clear in most of them, in both CTAs."""
    n, H, m = (74, 128, 1500) if whole else (40, 16, 1500)
    d = make([n], [m], H, seed=n)
    kw = dict(window=300, n_sink=70, out_dtype=torch.float32)
    assert (L.lib().ls_window_attention_workspace_size(1, n, H, n, 300, 1, 70) == 0) == whole
    q, args = d["q"].cuda(), (dev(d["start"]), dev(d["lens"]))
    want, wl = L.ls_window_attention(q, d["lat"].cuda(), *args, **kw)
    lat = d["lat"].clone()
    for i, r in enumerate([r for r in range(lat.shape[0]) if r >= m or 70 <= r < m - n - 300 + 1]):
        lat[r] = (float("nan"), float("inf"), -float("inf"))[i % 3]
    lat = lat.cuda()
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        o, z = L.ls_window_attention(q, lat, *args, **kw)
        bad += (o.view(torch.int32) != want.view(torch.int32)).sum() + (z.view(torch.int32) != wl.view(torch.int32)).sum()
    assert int(bad) == 0 and L.ls_device_status() == 0


@pytest.mark.parametrize("max_ctx", [1, 0])
def test_branches_that_are_not_finite_every_time(L, max_ctx):  # noqa: F811
    """The same for drafted rows: every odd token's row is not finite and seen by odd tokens alone, over several tiles of
    drafted rows."""
    n, H = 300, 16
    d = make([n], [200], H, seed=41, drafted=True)
    branches = [{i for i in range(n) if i % 2 == t % 2 and i <= t} for t in range(n)]
    mask, q, args = dev(tree_bits(branches, 5)), d["q"].cuda(), (dev(d["start"]), dev(d["lens"]))
    call = lambda lat: L.ls_tree_attention(q, lat, *args, mask, out_dtype=torch.float32, max_ctx=max_ctx)  # noqa: E731
    want, wl = call(d["lat"].cuda())
    lat = d["lat"].clone()
    for i in range(1, n, 2):
        lat[200 + i, (7 * i) % 512] = (float("nan"), float("inf"), -float("inf"))[i // 2 % 3]
    lat = lat.cuda()
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        o, z = call(lat)
        bad += (o[::2] != want[::2]).sum() + (z[::2] != wl[::2]).sum()
    assert int(bad) == 0 and L.ls_device_status() == 0
