"""Scored attention, rotary positions and paged attention as measured operators.

Three operators, each with a plain form in elementary torch operations (fp32,
fp64 for angles) and as the calls a user of the library makes:

* ``scored``: block-sparse attention over a plan whose scores are capped by a
  tanh, biased by distance and narrowed by a document and a prefix (or
  causal) mask, forward alone or with its gradients;
* ``rope``: rotary positions of Q and K (interleaved or half pairs, part of
  the head, one to three position axes, scaled frequencies), forward and
  backward, with the layout change from the projection's [B, S, H, D] to
  the attention's [B, H, S, D] in the same pass;
* ``paged``: attention of each sequence's new tokens over a paged cache, from
  a single token per sequence to long chunks.

A case is a dict of plain values.  Layouts (documents, lengths, page counts)
follow from the case alone; the seed makes tensor values and page orders.
"""

from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 64  # slots per logical block of a token sequence


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # the smallest video grid of the library's tests: launch latency counts
        {"name": "scored_fwd_video_tiny", "op": "scored", "train": False, "layout": "video", "grid": "5x6x10",
         "window": "3x3x3", "batch": 1, "heads": 2, "kv_heads": 2, "head_dim": 64, "softcap": 30.0, "bias": True,
         "mask": "frames", "prefix": 0, "doc_len": 0, "layout_seed": 1},
        # prompts packed into one row of 16384 tokens, with a padded tail: prefill or evaluation of short documents
        {"name": "scored_fwd_documents", "op": "scored", "train": False, "layout": "tokens", "tokens": 16384,
         "batch": 1, "heads": 16, "kv_heads": 16, "head_dim": 128, "softcap": 0.0, "bias": True, "mask": "docs",
         "prefix": 0, "doc_len": 900, "layout_seed": 2},
        # a fine-tuning batch of two short odd rows with grouped heads
        {"name": "scored_train_odd", "op": "scored", "train": True, "layout": "tokens", "tokens": 777, "batch": 2,
         "heads": 4, "kv_heads": 2, "head_dim": 64, "softcap": 20.0, "bias": False, "mask": "prefix", "prefix": 130,
         "doc_len": 0, "layout_seed": 3},
        # one long training row: a prefix seen by all, causal after it, capped scores, grouped heads
        {"name": "scored_train_prefix", "op": "scored", "train": True, "layout": "tokens", "tokens": 12289, "batch": 1,
         "heads": 16, "kv_heads": 4, "head_dim": 128, "softcap": 50.0, "bias": False, "mask": "prefix",
         "prefix": 1000, "doc_len": 0, "layout_seed": 4},
        # the full-occupancy video layout trained with frames in causal order and a decay over frames
        {"name": "scored_train_video", "op": "scored", "train": True, "layout": "video", "grid": "16x32x32",
         "window": "3x3x3", "batch": 1, "heads": 16, "kv_heads": 16, "head_dim": 128, "softcap": 30.0, "bias": True,
         "mask": "frames", "prefix": 0, "doc_len": 0, "layout_seed": 5},
        # one decoding step of 64 sequences
        {"name": "rope_decode", "op": "rope", "backward": False, "batch": 1, "slots": 64, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "rot_dim": 128, "interleaved": False, "sections": "64", "dtype": "bf16", "scaling": "yarn",
         "far": 100000, "layout_seed": 6},
        # Q and K of the 21x45x80 video grid: three axes, interleaved pairs
        {"name": "rope_video", "op": "rope", "backward": False, "batch": 1, "slots": 75600, "heads": 40,
         "kv_heads": 40, "head_dim": 128, "rot_dim": 128, "interleaved": True, "sections": "22x21x21",
         "dtype": "bf16", "scaling": "none", "far": 0, "layout_seed": 7},
        # the gradient on its way back to the projection: half pairs over part of an odd head size
        {"name": "rope_backward", "op": "rope", "backward": True, "batch": 2, "slots": 4099, "heads": 16,
         "kv_heads": 4, "head_dim": 96, "rot_dim": 64, "interleaved": False, "sections": "32", "dtype": "fp16",
         "scaling": "linear", "far": 0, "layout_seed": 8},
        # one token of one short sequence: latency
        {"name": "paged_one_token", "op": "paged", "seqs": 1, "q_lo": 1, "q_hi": 1, "kv_lo": 777, "kv_hi": 777,
         "heads": 16, "kv_heads": 4, "head_dim": 128, "page_slots": 16, "softcap": 30.0, "bias": False,
         "layout_seed": 9},
        # one decoding step of 64 sequences of very different lengths
        {"name": "paged_decode", "op": "paged", "seqs": 64, "q_lo": 1, "q_hi": 1, "kv_lo": 500, "kv_hi": 9000,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "page_slots": 64, "softcap": 0.0, "bias": False,
         "layout_seed": 10},
        # chunked prefill mixed with single tokens
        {"name": "paged_chunks", "op": "paged", "seqs": 5, "q_lo": 1, "q_hi": 700, "kv_lo": 900, "kv_hi": 20000,
         "heads": 16, "kv_heads": 4, "head_dim": 128, "page_slots": 32, "softcap": 50.0, "bias": True,
         "layout_seed": 11},
        # a chunk of 2048 tokens at the end of a 131072-token cache
        {"name": "paged_long_chunk", "op": "paged", "seqs": 1, "q_lo": 2048, "q_hi": 2048, "kv_lo": 131072,
         "kv_hi": 131072, "heads": 16, "kv_heads": 4, "head_dim": 128, "page_slots": 64, "softcap": 0.0,
         "bias": False, "layout_seed": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["scored", "scored", "rope", "paged"])
    seed = rng.randrange(1 << 30)
    if op == "scored":
        group = rng.choice([1, 1, 2, 4])
        kv = rng.choice([1, 2, 3, 4])
        c = {"op": op, "train": rng.random() < 0.6, "heads": kv * group, "kv_heads": kv,
             "head_dim": rng.choice([64, 128]), "softcap": rng.choice([0.0, 5.0, 20.0, 30.0, 50.0]),
             "bias": rng.random() < 0.5, "prefix": 0, "doc_len": 0, "layout_seed": seed}
        if rng.random() < 0.4:
            c.update(layout="video", batch=1, mask=rng.choice(["frames", "none"]),
                     grid="%dx%dx%d" % (_log_int(rng, 3, 16), _log_int(rng, 4, 32), _log_int(rng, 4, 32)),
                     window="%dx%dx%d" % (rng.choice([1, 2, 3]), rng.choice([2, 3, 5]), rng.choice([2, 3, 5])))
        else:
            c.update(layout="tokens", tokens=_log_int(rng, 1, 12000), mask=rng.choice(["prefix", "causal", "docs"]))
            c["batch"] = rng.choice([1, 1, 2, 3]) if c["tokens"] <= 4000 else 1
            if c["mask"] == "prefix":
                c["prefix"] = rng.randint(0, c["tokens"] if c["tokens"] <= 4000 else c["tokens"] // 8)
            if c["mask"] == "docs":
                c["doc_len"] = _log_int(rng, 1, max(1, c["tokens"]))
        return c
    if op == "rope":
        kv = rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([d, d, d // 2, d - 6])
        pairs = rot // 2
        axes = rng.choice([1, 1, 2, 3])
        cut = sorted(rng.randint(0, pairs) for _ in range(axes - 1))
        sections = "x".join(str(b - a) for a, b in zip([0] + cut, cut + [pairs]))
        c = {"op": op, "backward": rng.random() < 0.5, "batch": rng.choice([1, 2, 3]),
             "slots": _log_int(rng, 1, 40000), "heads": kv * rng.choice([1, 4]), "kv_heads": kv, "head_dim": d,
             "rot_dim": rot, "interleaved": rng.random() < 0.5, "sections": sections,
             "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
             "scaling": rng.choice(["none", "linear", "yarn"]), "far": rng.choice([0, 0, 100000, 2000000]),
             "layout_seed": seed}
        while work(c)["bytes"] > 3e9:
            c["slots"] //= 2
        return c
    kv = rng.choice([1, 2, 4, 8])
    q_hi = rng.choice([1, 1, _log_int(rng, 2, 2000)])
    seqs = _log_int(rng, 1, 64 if q_hi == 1 else 6)
    kv_hi = _log_int(rng, max(1, q_hi), max(q_hi, 60000 // (1 if seqs < 8 else 8)))
    c = {"op": op, "seqs": seqs, "q_lo": 1, "q_hi": min(q_hi, kv_hi), "kv_lo": max(1, kv_hi // 10),
         "kv_hi": kv_hi, "heads": kv * rng.choice([1, 2, 4, 8]), "kv_heads": kv,
         "head_dim": rng.choice([64, 128]), "page_slots": rng.choice([16, 32, 48, 64, 128]),
         "softcap": rng.choice([0.0, 0.0, 30.0, 50.0]), "bias": rng.random() < 0.4, "layout_seed": seed}
    while work(c)["flops"] > 2e12:
        c["q_hi"] = (c["q_hi"] + 1) // 2
    return c


# ----------------------------------------------------------------------------
# layouts (from the case alone)
# ----------------------------------------------------------------------------

def _dims(text):
    return [int(n) for n in text.split("x")]


def _video_layout(case):
    """(group [slots], frame [slots], graph [groups, groups]) of a T x H x W grid in 4x4x4 tiles."""
    T, H, W = _dims(case["grid"])
    nt, nh, nw = -(-T // 4), -(-H // 4), -(-W // 4)
    tile = np.arange(nt * nh * nw)
    tt, th, tw = tile // (nh * nw), tile // nw % nh, tile % nw
    inner = np.arange(64)
    t = tt[:, None] * 4 + inner // 16
    h = th[:, None] * 4 + inner // 4 % 4
    w = tw[:, None] * 4 + inner % 4
    valid = (t < T) & (h < H) & (w < W)
    group = np.where(valid, tile[:, None], -1).astype(np.int32).reshape(-1)
    frame = np.where(valid, t, 0).astype(np.int32).reshape(-1)

    def near(n, size):
        if n <= size:
            return np.ones((n, n), bool)
        first = np.clip(np.arange(n) - size // 2, 0, n - size)
        j = np.arange(n)
        return (j >= first[:, None]) & (j < first[:, None] + size)

    a, b, c = (near(n, s) for n, s in zip((nt, nh, nw), _dims(case["window"])))
    graph = a[tt[:, None], tt] & b[th[:, None], th] & c[tw[:, None], tw]
    return group, frame, graph


def _score_layout(case):
    """Groups, per-batch graphs and per-slot score arrays (NumPy) of a scored case."""
    B = case["batch"]
    rng = np.random.default_rng(case["layout_seed"])
    if case["layout"] == "video":
        group, frame, graph = _video_layout(case)
        out = {"group": group, "graphs": [graph], "pos": np.tile(frame, (B, 1)), "last": None, "doc": None}
        if case["mask"] == "frames":
            out["last"] = out["pos"]  # own frame and earlier ones
            # tiles of later frames only are not listed
            t0 = np.arange(graph.shape[0]) // (graph.shape[0] // -(-_dims(case["grid"])[0] // 4))
            out["graphs"] = [graph & (t0[None, :] <= t0[:, None])]
        return out
    N = case["tokens"]
    group = (np.arange(N) // BLOCK).astype(np.int32)
    nb = -(-N // BLOCK)
    pos = np.tile(np.arange(N, dtype=np.int32), (B, 1))
    blk = np.arange(nb)
    causal = blk[None, :] <= blk[:, None]
    out = {"group": group, "pos": pos, "last": pos, "doc": None}
    if case["mask"] == "causal":
        out["graphs"] = [causal]
    elif case["mask"] == "prefix":
        P = case["prefix"]
        out["last"] = np.maximum(pos, P - 1).astype(np.int32)
        out["graphs"] = [causal | (blk[None, :] * BLOCK < P)]
    else:
        docs, graphs = [], []
        for _ in range(B):
            doc = np.full(N, -1, np.int32)
            end = N - int(rng.integers(0, max(1, N // 16)))  # a padded tail: rows that attend nothing
            at = n = 0
            while at < end:
                size = 1 + int(rng.integers(0, 2 * case["doc_len"]))
                doc[at:min(end, at + size)] = n
                at, n = at + size, n + 1
            docs.append(doc)
            first = np.full(nb, N, np.int64)
            last = np.full(nb, -1, np.int64)
            real = doc >= 0
            np.minimum.at(first, group[real], doc[real])
            np.maximum.at(last, group[real], doc[real])
            graphs.append(causal & (last[None, :] >= first[:, None]))
        out["doc"] = np.stack(docs)
        out["graphs"] = graphs if B > 1 else graphs[:1]
    return out


def _pairs(case):
    """Allowed (query, key) pairs of one head, summed over the batch."""
    lay = _score_layout(case)
    total = 0
    for b in range(case["batch"]):
        graph = lay["graphs"][b if len(lay["graphs"]) > 1 else 0]
        if case["layout"] == "tokens":
            last, doc = lay["last"][b].astype(np.int64), None if lay["doc"] is None else lay["doc"][b]
            if doc is None:
                total += int(np.minimum(last + 1, case["tokens"]).sum())
            else:
                for n in np.unique(doc[doc >= 0]):
                    size = int((doc == n).sum())
                    total += size * (size + 1) // 2
            continue
        group, frame = lay["group"], lay["pos"][b]
        frames = _dims(case["grid"])[0]
        count = np.zeros((graph.shape[0], frames), np.int64)  # keys of a group, by frame
        real = group >= 0
        np.add.at(count, (group[real], frame[real]), 1)
        upto = np.cumsum(count, axis=1) if lay["last"] is not None else np.repeat(
            count.sum(1, keepdims=True), frames, axis=1)
        reach = graph.astype(np.int64) @ upto  # [group, frame]: keys that a query there may attend
        total += int(reach[group[real], frame[real]].sum())
    return total


def _slopes(heads):
    """Slopes of the distance bias: 2^(-8 (h + 1) / heads)."""
    return 2.0 ** (-8.0 * (np.arange(heads) + 1) / heads)


def _lens(case):
    """(new tokens, cache length with them) of each sequence."""
    rng = random.Random(case["layout_seed"])
    out = []
    for i in range(case["seqs"]):
        q = rng.randint(case["q_lo"], case["q_hi"]) if i % 3 != 1 else case["q_lo"]
        out.append((q, max(q, rng.randint(case["kv_lo"], case["kv_hi"]))))
    return out


def _freqs(case):
    """Radians per position of every pair, fp64."""
    pairs = case["rot_dim"] // 2
    f = np.zeros(pairs)
    at = 0
    for n in _dims(case["sections"]):  # each axis has its own ladder of frequencies
        if n:
            f[at:at + n] = 10000.0 ** (-np.arange(n) / n)
        at += n
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "yarn":
        # slow pairs are interpolated by 8, fast ones kept, a ramp between 1 and 32 turns over 4096 positions
        turns = 4096 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / 31.0, 0.0, 1.0)
        return f * keep + f / 8.0 * (1 - keep), 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def _rope_positions(case):
    """int32 [axes, slots]."""
    S, axes = case["slots"], len(_dims(case["sections"]))
    i = np.arange(S)
    if axes == 3:  # a grid 45 high and 80 wide
        pos = np.stack([i // 3600, i // 80 % 45, i % 80])
    elif axes == 2:
        pos = np.stack([i // 80, i % 80])
    else:
        pos = i[None]
    if case["far"]:
        rng = np.random.default_rng(case["layout_seed"])
        pos = pos + rng.integers(0, case["far"], size=(axes, S))
    return pos.astype(np.int32)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _randn(gen, shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _i32(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _tensors(case, seed):
    """The tensors of a case, the same for both forms and for ``exact``."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] == "scored":
        lay = _score_layout(case)
        B, H, Hk, D, S = case["batch"], case["heads"], case["kv_heads"], case["head_dim"], lay["group"].size
        # queries a little wider than unit variance, so that the cap and the softmax have something to do
        s = {"q": _randn(gen, (B, H, S, D), scale=1.5), "k": _randn(gen, (B, Hk, S, D)), "v": _randn(gen, (B, Hk, S, D))}
        if case["train"]:
            s["do"] = _randn(gen, (B, H, S, D))
        s["pos"], s["last"], s["doc"] = _i32(lay["pos"]), _i32(lay["last"]), _i32(lay["doc"])
        s["slopes"] = torch.tensor(_slopes(H), dtype=torch.float32, device=DEV) if case["bias"] else None
        s["group"] = torch.from_numpy(lay["group"].astype(np.int64)).to(DEV)
        s["graphs"] = [torch.from_numpy(g).to(DEV) for g in lay["graphs"]]
        return s, lay
    if case["op"] == "rope":
        B, S, H, Hk, D = (case[n] for n in ("batch", "slots", "heads", "kv_heads", "head_dim"))
        dt = DTYPES[case["dtype"]]
        f, m = _freqs(case)
        s = {"pos": _i32(_rope_positions(case)), "freqs": torch.from_numpy(f).to(DEV), "mscale": m}
        if case["backward"]:  # gradients as the attention leaves them
            s["q"], s["k"] = _randn(gen, (B, H, S, D), dt), _randn(gen, (B, Hk, S, D), dt)
        else:  # one projection's output, Q and K as views of it
            qkv = _randn(gen, (B, S, H + 2 * Hk, D), dt)
            s["q"], s["k"] = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hk].transpose(1, 2)
        return s, None
    lens = _lens(case)
    H, Hk, D, ps = (case[n] for n in ("heads", "kv_heads", "head_dim", "page_slots"))
    need = [-(-kv // ps) for _, kv in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=gen, device=DEV)
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n].to(torch.int32)
        at += n
    T = sum(q for q, _ in lens)
    s = {"q": _randn(gen, (T + 2, H, D), scale=1.5), "k": _randn(gen, (n_pages, ps, Hk, D)),
         "v": _randn(gen, (n_pages, ps, Hk, D)), "table": table, "lens": lens,
         "q_start": _i32(np.cumsum([0] + [q for q, _ in lens])), "kv_len": _i32([kv for _, kv in lens]),
         "slopes": torch.tensor(_slopes(H), dtype=torch.float32, device=DEV) if case["bias"] else None}
    # rows behind the last sequence stay as they were
    s["o"] = torch.zeros((T + 2, H, D), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros((T + 2, H), dtype=torch.float32, device=DEV)
    return s, None


def prepare(case, seed):
    s, lay = _tensors(case, seed)
    s["case"] = case
    if not own:
        return s
    import block_sparse_attention_bwd_b200 as sp

    if case["op"] == "scored":
        rows, cols = [0], []
        for g in lay["graphs"]:
            r, c = np.nonzero(g)
            counts = np.bincount(r, minlength=g.shape[0])
            for _ in range(case["heads"]):
                rows.extend((rows[-1] + np.cumsum(counts)).tolist())
                cols.append(c)
        n = lay["graphs"][0].shape[0]
        s["plan"] = sp.Plan(lay["group"], lay["group"], n, n, np.array(rows), np.concatenate(cols),
                            batch=case["batch"], heads=case["heads"], kv_heads=case["kv_heads"],
                            head_dim=case["head_dim"], graph_batches=len(lay["graphs"]))
        s["score"] = sp.Score(softcap=case["softcap"], slopes=s["slopes"], q_pos=s["pos"], k_pos=s["pos"],
                              q_last=s["last"], q_doc=s["doc"], k_doc=s["doc"])
    elif case["op"] == "paged":
        s["plan"] = sp.PagedPlan(heads=case["heads"], kv_heads=case["kv_heads"], head_dim=case["head_dim"],
                                 page_slots=case["page_slots"], max_seqs=case["seqs"], max_q=case["q_hi"],
                                 max_kv=max(kv for _, kv in s["lens"]), softcap=case["softcap"], slopes=s["slopes"])
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _allowed(s, b):
    """bool [S, S]: the pairs that batch entry b's graph and masks allow."""
    group = s["group"]
    graph = s["graphs"][b if len(s["graphs"]) > 1 else 0]
    real = group >= 0
    g = group.clamp(min=0)
    ok = graph[g][:, g] & real[:, None] & real[None, :]
    if s["last"] is not None:
        ok &= s["pos"][b][None, :] <= s["last"][b][:, None]
    if s["doc"] is not None:
        d = s["doc"][b]
        ok &= (d[:, None] == d[None, :]) & (d >= 0)[:, None]
    return ok


def _plain_scored(s):
    case = s["case"]
    B, H, Hk, D, cap = case["batch"], case["heads"], case["kv_heads"], case["head_dim"], case["softcap"]
    S = s["q"].shape[2]
    o = torch.empty((B, H, S, D), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((B, H, S), dtype=torch.float32, device=DEV)
    train = case["train"]
    if train:
        dq, dk = torch.empty_like(s["q"]), torch.zeros((B, Hk, S, D), device=DEV)
        dv = torch.zeros((B, Hk, S, D), device=DEV)
    scale = 1.0 / math.sqrt(D)
    kv_of = torch.arange(H, device=DEV) // (H // Hk)
    some = max(1, (1 << 29) // (S * S))  # heads at once: scores of at most 2 GB
    for b in range(B):
        ok = _allowed(s, b)
        dist = None
        if s["slopes"] is not None:
            p = s["pos"][b].float()
            dist = (p[:, None] - p[None, :]).abs()
        for heads in torch.arange(H, device=DEV).split(some):
            kv = kv_of[heads]
            q, k, v = s["q"][b, heads].float(), s["k"][b, kv].float(), s["v"][b, kv].float()
            z = (q @ k.mT) * scale
            t = None
            if cap:
                t = torch.tanh(z / cap)
                z = t * cap
            if dist is not None:
                z = z - s["slopes"][heads, None, None] * dist
            z = torch.where(ok, z, -math.inf)
            m = z.amax(dim=2, keepdim=True)
            m = torch.where(m == -math.inf, 0.0, m)
            p = torch.exp(z - m)
            l = p.sum(dim=2, keepdim=True)
            p = p / torch.where(l > 0, l, 1.0)
            o[b, heads] = (p @ v).to(o.dtype)
            lse[b, heads] = (m + torch.log(l))[..., 0]
            if not train:
                continue
            do = s["do"][b, heads].float()
            dv[b].index_add_(0, kv, p.mT @ do)
            dp = do @ v.mT
            ds = p * (dp - (p * dp).sum(dim=2, keepdim=True))
            if t is not None:
                ds = ds * (1 - t * t)
            dq[b, heads] = ((ds @ k) * scale).to(dq.dtype)
            dk[b].index_add_(0, kv, (ds.mT @ q) * scale)
    if not train:
        return o, lse
    return o, lse, dq, dk.to(torch.bfloat16), dv.to(torch.bfloat16)


def _angles(case, pos, freqs):
    """fp64 [slots, pairs]."""
    sections = _dims(case["sections"])
    axis = torch.from_numpy(np.repeat(np.arange(len(sections)), sections)).to(pos.device)
    return pos.double()[axis].T * freqs


def _rotate(x, cos, sin, rot, interleaved):
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    lo, hi = a * cos - b * sin, a * sin + b * cos
    r = torch.stack((lo, hi), dim=-1).flatten(-2) if interleaved else torch.cat((lo, hi), dim=-1)
    return torch.cat((r, x[..., rot:]), dim=-1)


def _plain_rope(s):
    case = s["case"]
    a = _angles(case, s["pos"], s["freqs"])
    if case["backward"]:
        a = -a
    cos, sin = (torch.cos(a) * s["mscale"]).float(), (torch.sin(a) * s["mscale"]).float()
    out = [_rotate(s[n].float(), cos, sin, case["rot_dim"], case["interleaved"]).to(s[n].dtype) for n in ("q", "k")]
    if case["backward"]:  # the projection's [B, S, H, D]
        out = [t.transpose(1, 2).contiguous() for t in out]
    return tuple(out)


def _plain_paged(s):
    case = s["case"]
    H, Hk, cap = case["heads"], case["kv_heads"], case["softcap"]
    o, lse = s["o"], s["lse"]
    at = 0
    for i, (nq, nkv) in enumerate(s["lens"]):
        pages = s["table"][i, :-(-nkv // case["page_slots"])].long()
        k = s["k"][pages].flatten(0, 1)[:nkv].float().transpose(0, 1)
        v = s["v"][pages].flatten(0, 1)[:nkv].float().transpose(0, 1)
        q = s["q"][at:at + nq].float().transpose(0, 1).unflatten(0, (Hk, H // Hk))
        q_pos = torch.arange(nkv - nq, nkv, device=DEV)
        k_pos = torch.arange(nkv, device=DEV)
        dist = (q_pos[:, None] - k_pos[None, :]).float()
        some = max(1, (1 << 30) // (H // Hk * nq * nkv))  # K/V heads at once: scores of at most 4 GB
        for kv in range(0, Hk, some):
            qs, ks, vs = q[kv:kv + some], k[kv:kv + some, None], v[kv:kv + some, None]
            z = torch.matmul(qs, ks.mT) / math.sqrt(case["head_dim"])
            if cap:
                z = torch.tanh(z / cap) * cap
            if s["slopes"] is not None:
                z = z - s["slopes"].unflatten(0, (Hk, -1))[kv:kv + some, :, None, None] * dist
            z = torch.where(dist >= 0, z, -math.inf)
            m = z.amax(dim=3, keepdim=True)
            p = torch.exp(z - m)
            l = p.sum(dim=3, keepdim=True)
            heads = slice(kv * (H // Hk), (kv + some) * (H // Hk))
            o[at:at + nq, heads] = (torch.matmul(p, vs) / l).flatten(0, 1).transpose(0, 1).to(o.dtype)
            lse[at:at + nq, heads] = (m + torch.log(l))[..., 0].flatten(0, 1).T
        at += nq
    return o, lse


def run(state):
    case = state["case"]
    if not own:
        return {"scored": _plain_scored, "rope": _plain_rope, "paged": _plain_paged}[case["op"]](state)
    import block_sparse_attention_bwd_b200 as sp

    s = state
    if case["op"] == "scored":
        o, lse = sp.spattn_fwd_scored(s["q"], s["k"], s["v"], s["plan"], s["score"])
        if not case["train"]:
            return o, lse
        return (o, lse) + tuple(sp.spattn_bwd_scored(s["q"], s["k"], s["v"], o, lse, s["do"], s["plan"], s["score"]))
    if case["op"] == "rope":
        kw = dict(rot_dim=case["rot_dim"], interleaved=case["interleaved"], sections=_dims(case["sections"]),
                  mscale=s["mscale"])
        if not case["backward"]:
            return sp.rope(s["q"], s["k"], s["pos"], s["freqs"], **kw)
        B, H, S, D = s["q"].shape
        dq = torch.empty((B, S, H, D), dtype=s["q"].dtype, device=DEV)
        dk = torch.empty((B, S, case["kv_heads"], D), dtype=s["q"].dtype, device=DEV)
        sp.rope_bwd(s["q"], s["k"], s["pos"], s["freqs"], dq=dq.transpose(1, 2), dk=dk.transpose(1, 2), **kw)
        return dq, dk
    return sp.spattn_paged_fwd(s["q"], s["k"], s["v"], s["table"], s["q_start"], s["kv_len"], s["plan"], o=s["o"],
                               lse=s["lse"])


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    H, Hk, D = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "scored":
        lay = _score_layout(case)
        S = lay["group"].size
        q, kv, rows = (case["batch"] * S * n for n in (H * D, Hk * D, H))
        pairs = _pairs(case) * H
        if not case["train"]:  # q, k, v in; o, lse out
            return {"bytes": 2 * (2 * q + 2 * kv) + 4 * rows, "flops": 4 * D * pairs}
        # q, k, v, do in; o, lse, dq, dk, dv out; two products forward, five backward
        return {"bytes": 2 * (4 * q + 4 * kv) + 4 * rows, "flops": 14 * D * pairs}
    if case["op"] == "rope":
        n = case["batch"] * case["slots"] * (H + Hk)
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 2 * size * n * D + 4 * len(_dims(case["sections"])) * case["slots"] + 8 * (case["rot_dim"] // 2),
                "flops": 3 * n * case["rot_dim"]}
    lens = _lens(case)
    T, cached = sum(q for q, _ in lens), sum(kv for _, kv in lens)
    pairs = sum(q * kv - q * (q - 1) // 2 for q, kv in lens) * H
    return {"bytes": 2 * (2 * T * H * D + 2 * cached * Hk * D) + 4 * T * H, "flops": 4 * D * pairs}


# ----------------------------------------------------------------------------
# 64-bit values, from the definitions, row block by row block
# ----------------------------------------------------------------------------

def _rows64(q, k, v, z_of, do=None):
    """Softmax attention and its gradients of one head in fp64, over blocks of 2048 query rows.

    ``z_of(raw, rows)`` gives (scores with -inf where masked, d score / d raw).
    """
    n, D = q.shape
    o, lse = torch.zeros_like(q), torch.zeros(n, dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a in range(0, n, 2048):
        rows = slice(a, min(n, a + 2048))
        z, slope = z_of(q[rows] @ k.T, rows)
        lse[rows] = torch.logsumexp(z, dim=1)
        w = torch.where(torch.isinf(z), 0.0, torch.exp(z - lse[rows, None]))
        o[rows] = w @ v
        if do is not None:
            g = do[rows] @ v.T
            ds = w * (g - (do[rows] * o[rows]).sum(1, keepdim=True)) * slope
            dq[rows] = ds @ k
            dk += ds.T @ q[rows]
            dv += w.T @ do[rows]
    return o, lse, dq, dk, dv


def _capped64(raw, D, cap):
    x = raw / math.sqrt(D)
    if not cap:
        return x, 1.0 / math.sqrt(D)
    y = cap * torch.tanh(x / cap)
    return y, (1 - (y / cap) ** 2) / math.sqrt(D)


def _exact_scored(case, s):
    B, H, Hk, D = case["batch"], case["heads"], case["kv_heads"], case["head_dim"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    do = s["do"].double() if case["train"] else None
    out = [torch.zeros_like(q), torch.zeros(q.shape[:3], dtype=torch.float64, device=DEV), torch.zeros_like(q),
           torch.zeros_like(k), torch.zeros_like(v)]
    real = s["group"] >= 0
    for b in range(B):
        graph = s["graphs"][b if len(s["graphs"]) > 1 else 0]
        pos = s["pos"][b].double()
        for h in range(H):
            def z_of(raw, rows):
                y, slope = _capped64(raw, D, case["softcap"])
                if case["bias"]:
                    y = y - float(s["slopes"][h]) * torch.abs(pos[rows, None] - pos[None, :])
                ban = ~(real[rows, None] & real[None, :])
                ban |= ~graph[s["group"][rows].clamp(min=0)][:, s["group"].clamp(min=0)]
                if s["last"] is not None:
                    ban |= s["pos"][b][None, :] > s["last"][b][rows, None]
                if s["doc"] is not None:
                    ban |= (s["doc"][b][rows, None] != s["doc"][b][None, :]) | (s["doc"][b][rows, None] < 0)
                return y.masked_fill(ban, -math.inf), slope

            hk = h * Hk // H
            r = _rows64(q[b, h], k[b, hk], v[b, hk], z_of, None if do is None else do[b, h])
            for t, x in zip(out[:3], r[:3]):
                t[b, h] = x
            out[3][b, hk] += r[3]
            out[4][b, hk] += r[4]
    return tuple(out) if case["train"] else tuple(out[:2])


def _exact_rope(case, s):
    pos = s["pos"].cpu().numpy().astype(np.float64)
    f, m = _freqs(case)
    cut = np.cumsum([0] + _dims(case["sections"]))
    ang = np.concatenate([np.outer(pos[i], f[cut[i]:cut[i + 1]]) for i in range(len(pos))], axis=1)
    turn = torch.polar(torch.full(ang.shape, float(m), dtype=torch.float64), torch.from_numpy(ang)).to(DEV)
    if case["backward"]:
        turn = turn.conj()
    out = []
    for n in ("q", "k"):
        y = s[n].double().clone()
        r = case["rot_dim"]
        i = torch.arange(r // 2, device=DEV)
        lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
        c = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * turn
        y[..., lo], y[..., hi] = c.real.clone(), c.imag.clone()
        out.append(y.transpose(1, 2).contiguous() if case["backward"] else y)
    return tuple(out)


def _exact_paged(case, s):
    o, lse = s["o"].double(), s["lse"].double()
    H, Hk, D, ps = (case[n] for n in ("heads", "kv_heads", "head_dim", "page_slots"))
    at = 0
    for i, (nq, nkv) in enumerate(s["lens"]):
        j = torch.arange(nkv, device=DEV)
        page, off = s["table"][i].long()[j // ps], j % ps
        for h in range(H):
            def z_of(raw, rows):
                y, slope = _capped64(raw, D, case["softcap"])
                me = torch.arange(nkv - nq, nkv, device=DEV)[rows]
                if case["bias"]:
                    y = y - float(s["slopes"][h]) * (me[:, None] - j[None, :]).double()
                return y.masked_fill(j[None, :] > me[:, None], -math.inf), slope

            hk = h * Hk // H
            r = _rows64(s["q"][at:at + nq, h].double(), s["k"][page, off, hk].double(), s["v"][page, off, hk].double(),
                        z_of)
            o[at:at + nq, h], lse[at:at + nq, h] = r[0], r[1]
        at += nq
    return o, lse


def exact(case, seed):
    if work(case)["flops"] > 6e12:  # fp64 products of a larger case take too long
        return None
    s, _ = _tensors(case, seed)
    return {"scored": _exact_scored, "rope": _exact_rope, "paged": _exact_paged}[case["op"]](case, s)
