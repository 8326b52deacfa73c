"""Workloads of the attention-side operators around the sparse attention, with their plain forms.

* window attention: every query attends to the first rows of its sequence
  (sinks) and to a sliding or block-aligned window of the latest rows of the
  latent cache (576-element rows: the key of every head; the first 512
  elements are the value);
* tree attention: drafted tokens attend to their sequence's whole context and,
  among the drafted rows that follow it, to their own branch;
* norm and rotation: the norm of the query heads and of the key, the position
  rotation, and the write into the (bf16 or fp8) cache rows, in one pass.

`own` chooses between the plain form (elementary torch operations in 32 bits)
and the package's calls.  Cases are plain dicts; `_lens` derives the ragged
lengths of a batch from the case alone, so every seed has the same shapes.
"""

import math
import random

import torch

own = False

LATENT, VALUE = 576, 512


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def listed():
    return [
        # One decoded token of one conversation: the smallest call, all latency.
        dict(name="window_decode_1", op="window", B=1, n=1, n_min=1, H=128, kv=32768, kv_min=32768, window=512,
             align=1, n_sink=4, mix=1),
        # A decode step of a batch of conversations of very different ages, some younger than the window.
        dict(name="window_decode_64", op="window", B=64, n=1, n_min=1, H=128, kv=32768, kv_min=3, window=512,
             align=1, n_sink=4, mix=2),
        # A prefill chunk of one long conversation: the largest call.
        dict(name="window_prefill_4096", op="window", B=1, n=4096, n_min=4096, H=128, kv=131072, kv_min=131072,
             window=512, align=1, n_sink=4, mix=3),
        # Ragged prefill pieces on a rank that holds 16 heads, with the block window of the bucket search.
        dict(name="window_blocks_h16", op="window", B=6, n=701, n_min=1, H=16, kv=9000, kv_min=900, window=1,
             align=512, n_sink=4, mix=4),
        # Five drafted tokens on a prompt of a few lines.
        dict(name="tree_short", op="tree", B=1, n=5, n_min=5, H=128, kv=100, kv_min=100, mix=5),
        # Sixteen drafted tokens of one long conversation: few query rows over a long axis.
        dict(name="tree_16_over_32768", op="tree", B=1, n=16, n_min=16, H=128, kv=32768, kv_min=32768, mix=6),
        # A verification step of a batch on a rank that holds 16 heads: bound by the cache's bytes.
        dict(name="tree_32x8_h16", op="tree", B=32, n=8, n_min=1, H=16, kv=16384, kv_min=1000, mix=7),
        # A verification step with wide trees and all heads: bound by the products.
        dict(name="tree_8x48", op="tree", B=8, n=48, n_min=33, H=128, kv=12000, kv_min=4000, mix=8),
        # One decoded token's indexer query heads and key.
        dict(name="norm_decode_1", op="norm", T=1, Hq=32, d=128, q_norm="rms", k_norm="layer", norm_dim=128,
             rope_off=0, rope=64, interleaved=False, fp8=False, rows=4096, pos_max=131072, mix=9),
        # A decode step's indexer queries and keys, written as fp8 codes and scales.
        dict(name="norm_decode_64_fp8", op="norm", T=64, Hq=32, d=128, q_norm="none", k_norm="layer", norm_dim=128,
             rope_off=0, rope=64, interleaved=False, fp8=True, rows=65536, pos_max=10485760, mix=10),
        # A prefill chunk's indexer queries and keys as fp8.
        dict(name="norm_prefill_4096_fp8", op="norm", T=4096, Hq=32, d=128, q_norm="rms", k_norm="layer",
             norm_dim=128, rope_off=0, rope=64, interleaved=False, fp8=True, rows=8192, pos_max=131072, mix=11),
        # A prefill chunk's absorbed queries (rotated part last) and latent rows (normed first 512) of the attention.
        dict(name="norm_latent_2048", op="norm", T=2048, Hq=128, d=576, q_norm="none", k_norm="rms", norm_dim=512,
             rope_off=512, rope=64, interleaved=True, fp8=False, rows=4096, pos_max=131072, mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    mix = rng.randrange(100, 1 << 30)
    op = rng.choice(("window", "tree", "norm"))
    if op == "window":
        H = rng.choice((1, 8, 16, 24, 32, 64, 128))
        if rng.random() < 0.5:                        # decode: a token or a few for each sequence
            B, n = _log(rng, 1, 96), rng.choice((1, 1, 1, 2, 3))
        else:                                         # prefill pieces
            B = rng.randint(1, 6)
            n = _log(rng, 4, min(4096, max(8, 4096 * 128 // (2 * B * max(H, 32)))))
        kv = _log(rng, max(n, 16), 65536 // (1 if B < 8 else 4))
        window, align = (1, 512) if rng.random() < 0.3 else (_log(rng, 1, 512), 1)
        return dict(op=op, B=B, n=n, n_min=1, H=H, kv=kv, kv_min=max(n, kv // 8, 1), window=window, align=align,
                    n_sink=rng.choice((0, 1, 4, 4, 5, 16)), mix=mix)
    if op == "tree":
        H = rng.choice((8, 16, 32, 64, 128))
        B, n = _log(rng, 1, 24), _log(rng, 1, 80)
        n = max(1, min(n, 8 * 48 * 128 // (2 * B * H)))
        kv = _log(rng, 16, max(64, min(40000, 8 * 48 * 128 * 6000 // (B * n * H), 400000 // B)))
        return dict(op=op, B=B, n=n, n_min=max(1, n // 2), H=H, kv=kv, kv_min=rng.choice((0, kv // 4, kv)), mix=mix)
    latent = rng.random() < 0.3
    T = _log(rng, 1, 1500 if latent else 4096)
    d = 576 if latent else rng.choice((64, 128, 128, 192))
    norm_dim = 512 if latent else d
    rope = 64 if latent else rng.choice((32, 64))
    return dict(op=op, T=T, Hq=rng.choice((16, 128) if latent else (1, 8, 32, 64)), d=d,
                q_norm="none" if latent else rng.choice(("rms", "layer", "none")),
                k_norm="rms" if latent else rng.choice(("rms", "layer")), norm_dim=norm_dim,
                rope_off=512 if latent else rng.choice((0, d - rope)), rope=rope,
                interleaved=rng.random() < 0.5, fp8=(not latent) and rng.random() < 0.5, rows=T + rng.randint(0, 4096),
                pos_max=rng.choice((4096, 131072, 10485760)), mix=mix)


def _lens(case):
    """(query tokens, cache rows) of each sequence: the first has the most of both, the others are spread."""
    r = random.Random(case["mix"])
    ns = [case["n"]] + [r.randint(case["n_min"], case["n"]) for _ in range(case["B"] - 1)]
    kv = [case["kv"]] + [r.randint(case["kv_min"], case["kv"]) for _ in range(case["B"] - 1)]
    if case["op"] == "window":                        # a sequence's rows include those of its query tokens
        kv = [max(a, b) for a, b in zip(ns, kv)]
    return ns, kv


def _lo(case, p):
    """First row of the window of the token at position p."""
    return max(0, (p - case["window"] + 1) // case["align"] * case["align"])


def _tree(case):
    """For each sequence, for each drafted token, the set of drafted tokens that it sees: its branch and itself."""
    r = random.Random(case["mix"] + 1)
    out = []
    for n in _lens(case)[0]:
        seen = []
        for i in range(n):
            parent = r.randint(max(-1, i - 6), i - 1)
            seen.append((seen[parent] if parent >= 0 else frozenset()) | {i})
        out.append(seen)
    return out


def work(case):
    if case["op"] == "norm":
        T, Hq, d = case["T"], case["Hq"], case["d"]
        heads = T * (Hq + 1)
        out = heads * (d + 4) if case["fp8"] else heads * 2 * d
        return {"bytes": heads * 2 * d + out + 16 * T, "flops": heads * (6 * d + 3 * case["rope"])}
    ns, kv = _lens(case)
    H, T = case["H"], sum(ns)
    seen = rows = 0
    if case["op"] == "window":
        for n, m in zip(ns, kv):
            for p in range(m - n, m):
                lo = _lo(case, p)
                seen += p + 1 - lo + min(case["n_sink"], lo)
            lo = _lo(case, m - n)
            rows += m - lo + min(case["n_sink"], lo)
    else:
        for n, m, tree in zip(ns, kv, _tree(case)):
            seen += n * m + sum(len(s) for s in tree)
            rows += m + n
    return {"bytes": T * H * (LATENT * 2 + VALUE * 2 + 4) + rows * LATENT * 2,
            "flops": 2.0 * seen * H * (LATENT + VALUE)}


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + case["mix"])

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    def dev(v, dtype):
        return torch.tensor(v, dtype=dtype, device="cuda")

    s = {"case": dict(case)}
    if case["op"] == "norm":
        T, Hq, d = case["T"], case["Hq"], case["d"]
        # the queries and the key of a token lie side by side, as one projection leaves them
        qk = randn(T, (Hq + 1) * d) * 3
        s["q"] = qk[:, :Hq * d].unflatten(1, (Hq, d))
        s["k"] = qk[:, Hq * d:].unflatten(1, (1, d))
        s["q_weight"] = 1 + 0.2 * torch.randn(case["norm_dim"], generator=g, device="cuda")
        s["k_weight"] = 1 + 0.2 * torch.randn(case["norm_dim"], generator=g, device="cuda")
        s["k_bias"] = 0.1 * torch.randn(case["norm_dim"], generator=g, device="cuda")
        s["pos"] = torch.randint(0, case["pos_max"], (T,), generator=g, device="cuda")
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, case["rope"], 2, device="cuda", dtype=torch.float64)
                                     / case["rope"])).float()
        s["slots"] = torch.randperm(case["rows"], generator=g, device="cuda")[:T].contiguous()
        cache = randn(case["rows"], d)
        s["k_scale"] = None
        if case["fp8"]:
            cache = cache.to(torch.float8_e4m3fn)
            s["k_scale"] = torch.rand(case["rows"], generator=g, device="cuda")
        s["k_cache"] = cache
        return s

    ns, kv = _lens(case)
    T, H = sum(ns), case["H"]
    extra = ns if case["op"] == "tree" else [0] * len(ns)
    cap = [m + e + 5 for m, e in zip(kv, extra)]      # each sequence's rows, and a few unused ones behind them
    off = [sum(cap[:i]) for i in range(len(cap))]
    s["ns"], s["kv"] = ns, kv
    # latent rows share a direction, as trained latents do; logits have a deviation of about 2
    s["latent"] = randn(sum(cap), LATENT) + 0.7 * randn(LATENT)
    s["q"] = randn(T, H, LATENT) * 2
    s["scale"] = LATENT ** -0.5
    s["q_start"] = dev([sum(ns[:i]) for i in range(len(ns) + 1)], torch.int32)
    s["kv_len"] = dev(kv, torch.int32)
    s["row_off"] = dev(off, torch.int64)
    s["seq"] = dev([b for b, n in enumerate(ns) for _ in range(n)], torch.int64)
    s["tok"] = dev([i for n in ns for i in range(n)], torch.int64)
    if case["op"] == "tree":
        words = (max(ns) + 63) // 64
        bits = []
        for tree in _tree(case):
            for seen in tree:
                v = [sum(1 << (j - 64 * w) for j in seen if 64 * w <= j < 64 * w + 64) for w in range(words)]
                bits.append([x - (1 << 64) if x >> 63 else x for x in v])
        s["tree_mask"] = dev(bits, torch.int64)
    return s


# --------------------------------------------------------------------------- #
# one pass
# --------------------------------------------------------------------------- #
def _softmax_rows(logits, seen):
    """Softmax weights and log-sum-exp along the last axis over the places `seen`; a row that sees nothing weighs 0."""
    logits = torch.where(seen, logits, torch.full_like(logits, -math.inf))
    top = logits.amax(dim=-1, keepdim=True)
    ref = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(logits - ref)
    den = e.sum(dim=-1, keepdim=True)
    lse = (ref + torch.log(den)).squeeze(-1)
    return e / torch.where(den == 0, torch.ones_like(den), den), lse


def _window_plain(s):
    case = s["case"]
    W = case["window"] + case["align"] - 1
    n_of = s["q_start"][1:] - s["q_start"][:-1]
    p = (s["kv_len"] - n_of).long()[s["seq"]] + s["tok"]                    # [T]
    lo = ((p - case["window"] + 1).div(case["align"], rounding_mode="floor") * case["align"]).clamp(min=0)
    sinks = torch.arange(case["n_sink"], device=p.device)[None, :].expand(p.numel(), -1)
    near = lo[:, None] + torch.arange(W, device=p.device)[None, :]
    rows = torch.cat([sinks, near], dim=1)                                  # [T, n_sink + W]
    seen = torch.cat([sinks < lo[:, None], near <= p[:, None]], dim=1)
    rows = torch.where(seen, rows + s["row_off"][s["seq"]][:, None], torch.zeros_like(rows))
    kv = s["latent"][rows].float()                                          # [T, n_sink + W, 576]
    logits = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * s["scale"]  # [T, H, n_sink + W]
    weights, lse = _softmax_rows(logits, seen[:, None, :])
    return torch.matmul(weights, kv[:, :, :VALUE]).to(torch.bfloat16), lse


def _tree_plain(s):
    case = s["case"]
    B, H, n, m = case["B"], case["H"], max(s["ns"]), max(s["kv"])
    dev = s["q"].device
    i = torch.arange(n, device=dev)
    j = torch.arange(m, device=dev)
    n_of = (s["q_start"][1:] - s["q_start"][:-1]).long()[:, None]           # [B, 1]
    m_of = s["kv_len"].long()[:, None]
    tok = torch.where(i[None, :] < n_of, s["q_start"][:-1].long()[:, None] + i[None, :], torch.zeros_like(n_of))
    # context rows, then drafted rows, each padded to the longest
    near = torch.cat([torch.where(j[None, :] < m_of, j[None, :], torch.zeros_like(m_of)),
                      torch.where(i[None, :] < n_of, m_of + i[None, :], torch.zeros_like(m_of))], dim=1)
    kv = s["latent"][near + s["row_off"][:, None]].float()                  # [B, m + n, 576]
    q = s["q"][tok].float()                                                 # [B, n, H, 576]
    branch = (s["tree_mask"][tok][:, :, i // 64] >> (i % 64)) & 1           # [B, n, n]
    branch = (branch == 1) & (i[None, None, :] < n_of[:, :, None])
    seen = torch.cat([(j[None, None, :] < m_of[:, :, None]).expand(B, n, m), branch], dim=2)
    logits = torch.matmul(q.reshape(B, n * H, LATENT), kv.transpose(1, 2)) * s["scale"]
    weights, lse = _softmax_rows(logits.view(B, n, H, m + n), seen[:, :, None, :])
    out = torch.matmul(weights.view(B, n * H, m + n), kv[:, :, :VALUE]).view(B, n, H, VALUE)
    return out[s["seq"], s["tok"]].to(torch.bfloat16), lse[s["seq"], s["tok"]]


def _normed(x, kind, dim, weight, bias):
    """x [.., d] float: its first `dim` elements normed, the others as they are."""
    if kind == "none":
        return x
    a = x[..., :dim]
    if kind == "layer":
        a = a - a.mean(dim=-1, keepdim=True)
    a = a * torch.rsqrt((a * a).mean(dim=-1, keepdim=True) + 1e-6) * weight
    if bias is not None:
        a = a + bias
    return torch.cat([a, x[..., dim:]], dim=-1)


def _rotated(x, case, cos, sin):
    """x [T, h, d]: elements rope_off .. rope_off + rope - 1 rotated by the token's angles (cos, sin [T, 1, rope / 2])."""
    o, r = case["rope_off"], case["rope"]
    mid = x[..., o:o + r]
    if case["interleaved"]:
        a, b = mid[..., 0::2], mid[..., 1::2]
        mid = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = mid[..., :r // 2], mid[..., r // 2:]
        mid = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([x[..., :o], mid, x[..., o + r:]], dim=-1)


def _codes(y):
    """(e4m3 codes, scale) of the rows of y: the largest magnitude of a row becomes 448."""
    top = y.abs().amax(dim=-1, keepdim=True)
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    return (y / scale).to(torch.float8_e4m3fn), scale.squeeze(-1)


def _norm_plain(s):
    case = s["case"]
    # angles of far positions need 64 bits: 10 M positions leave 32-bit ones wrong in the first digit
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()[None, :]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    q = _rotated(_normed(s["q"].float(), case["q_norm"], case["norm_dim"], s["q_weight"], None), case, cos, sin)
    k = _rotated(_normed(s["k"].float(), case["k_norm"], case["norm_dim"], s["k_weight"],
                         s["k_bias"] if case["k_norm"] == "layer" else None), case, cos, sin)[:, 0]
    if case["fp8"]:
        q8, q_scale = _codes(q)
        k8, k_scale = _codes(k)
        s["k_cache"].view(torch.uint8)[s["slots"]] = k8.view(torch.uint8)
        s["k_scale"][s["slots"]] = k_scale
        return q8, q_scale, s["k_cache"], s["k_scale"]
    s["k_cache"][s["slots"]] = k.to(torch.bfloat16)
    return q.to(torch.bfloat16), s["k_cache"]


def run(state):
    s, case = state, state["case"]
    if own:
        import sparse_attention_indexer_lightning_b200 as ls
        if case["op"] == "window":
            return ls.ls_window_attention(s["q"], s["latent"], s["q_start"], s["kv_len"], row_off=s["row_off"],
                                          window=case["window"], align=case["align"], n_sink=case["n_sink"],
                                          max_q=max(s["ns"]), scale=s["scale"])
        if case["op"] == "tree":
            return ls.ls_tree_attention(s["q"], s["latent"], s["q_start"], s["kv_len"], s["tree_mask"],
                                        row_off=s["row_off"], max_q=max(s["ns"]), max_ctx=max(s["kv"]),
                                        scale=s["scale"])
        q, q_scale, k_cache, k_scale = ls.ls_norm_rope(
            s["q"], s["k"], s["pos"], s["inv_freq"], q_norm=case["q_norm"], k_norm=case["k_norm"],
            norm_dim=case["norm_dim"], q_weight=s["q_weight"] if case["q_norm"] != "none" else None,
            k_weight=s["k_weight"], k_bias=s["k_bias"] if case["k_norm"] == "layer" else None, eps=1e-6,
            rope_off=case["rope_off"], interleaved=case["interleaved"], k_cache=s["k_cache"], k_scale=s["k_scale"],
            slots=s["slots"])
        return (q, q_scale, k_cache, k_scale) if case["fp8"] else (q, k_cache)
    return {"window": _window_plain, "tree": _tree_plain, "norm": _norm_plain}[case["op"]](s)


# --------------------------------------------------------------------------- #
# the definition in 64 bits
# --------------------------------------------------------------------------- #
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _norm_exact(case, s)
    ns, kv = _lens(case)
    H = case["H"]
    outs, lses = [], []
    for b, (n, m) in enumerate(zip(ns, kv)):
        first = int(s["q_start"][b])
        base = int(s["row_off"][b])
        tree = _tree(case)[b] if case["op"] == "tree" else None
        step = max(1, min(32, 40_000_000 // (H * (m + n)))) if tree is not None else 32
        for t0 in range(0, n, step):
            ts = list(range(t0, min(n, t0 + step)))
            if tree is not None:
                rows = list(range(m + n))
                seen = torch.zeros(len(ts), m + n, dtype=torch.bool)
                seen[:, :m] = True
                for a, t in enumerate(ts):
                    seen[a, [m + x for x in tree[t]]] = True
            else:
                ps = [m - n + t for t in ts]
                lo = _lo(case, ps[0])
                rows = sorted(set(range(min(case["n_sink"], ps[-1] + 1))) | set(range(lo, ps[-1] + 1)))
                at = torch.tensor(rows)
                seen = torch.stack([(at <= p) & ((at < case["n_sink"]) | (at >= _lo(case, p))) for p in ps])
            c = s["latent"][torch.tensor(rows, device="cuda") + base].double()
            q = s["q"][first + t0:first + t0 + len(ts)].double()
            z = torch.einsum("thd,rd->thr", q, c) * s["scale"]
            z.masked_fill_(~seen.cuda()[:, None, :], -math.inf)
            lse = torch.logsumexp(z, dim=-1)
            w = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[..., None])
            outs.append(torch.einsum("thr,rv->thv", w, c[:, :VALUE]))
            lses.append(lse)
    return torch.cat(outs), torch.cat(lses)


def _norm_exact(case, s):
    d, o, r = case["d"], case["rope_off"], case["rope"]
    half = r // 2
    # the rotation as a full matrix of index and sign: y = x * C + x[partner] * S
    i = torch.arange(r, device="cuda")
    pair = i // 2 if case["interleaved"] else i % half
    second = (i % 2 == 1) if case["interleaved"] else (i >= half)
    if case["interleaved"]:
        partner = torch.where(second, i - 1, i + 1)
    else:
        partner = torch.where(second, i - half, i + half)
    turns = s["pos"].double()[:, None] * s["inv_freq"].double()[pair][None, :]
    C, S = torch.cos(turns)[:, None, :], torch.where(second, 1.0, -1.0).double() * torch.sin(turns)[:, None, :]
    res = []
    for x, kind, weight, bias in ((s["q"], case["q_norm"], s["q_weight"], None),
                                  (s["k"], case["k_norm"], s["k_weight"], s["k_bias"])):
        y = x.double().clone()
        nd = case["norm_dim"]
        if kind != "none":
            mean = y[..., :nd].sum(-1, keepdim=True) / nd if kind == "layer" else 0.0
            dev = y[..., :nd] - mean
            std = torch.sqrt((dev ** 2).sum(-1, keepdim=True) / nd + 1e-6)
            y[..., :nd] = dev / std * weight.double()
            if kind == "layer" and bias is not None:
                y[..., :nd] += bias.double()
        part = y[..., o:o + r].clone()
        y[..., o:o + r] = part * C + part[..., partner] * S
        res.append(y)
    q, k = res[0], res[1][:, 0]
    if not case["fp8"]:
        cache = s["k_cache"].double()
        cache[s["slots"]] = k
        return q, cache
    # codes are compared through the values they stand for before their rounding
    q_scale = q.abs().amax(-1) / 448.0
    k_scale = k.abs().amax(-1) / 448.0
    cache, scales = s["k_cache"].double(), s["k_scale"].double()
    cache[s["slots"]] = k / k_scale[:, None]
    scales[s["slots"]] = k_scale
    return q / q_scale[..., None], q_scale, cache, scales
