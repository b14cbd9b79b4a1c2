"""Workloads of the operators around normalised queries and keys and of shared
prefixes: norms of queries and keys for each head with the position rotation (and
their gradient), appending to a paged cache with both applied on the way, and
attention of a batch whose sequences share long prefixes.

Each operator has a plain form of elementary torch operations (``own`` false) and
the framework's call (``own`` true).  The cache of one layer is three pools:
k and v pages [pages][kv heads][page tokens][head dim] in bf16, and pooled block
keys [pages][kv heads][head dim] in fp32, a block's mean key standing in the slot
of the block's last page.  Token p of sequence b lies in page
``table[b, p // page]`` at offset ``p % page``.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _norm(name, tokens, hq, hkv, d, rot, interleaved, grad, wide, far):
    return {"name": name, "op": "norm", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "interleaved": interleaved, "grad": grad, "wide": wide, "far": far}


def _append(name, seqs, new, ctx, hq, hkv, d, rot, interleaved, page, block, norm, shift, mix):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "ctx": ctx, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "interleaved": interleaved, "page": page, "block": block, "norm": norm, "shift": shift, "mix": mix}


def _shared(name, groups, seqs, new, prefix, tail, hq, hkv, d, page, mix):
    return {"name": name, "op": "shared", "groups": groups, "seqs": seqs, "new": new, "prefix": prefix, "tail": tail,
            "hq": hq, "hkv": hkv, "d": d, "page": page, "mix": mix}


def listed():
    return [
        # a training step's q and k at the 32K shape, whole heads rotated
        _norm("norm_train", 32768, 32, 32, 128, 128, False, False, False, 32768),
        # its gradient, with those of the weights: odd length, grouped heads, half of each head rotated, far positions
        _norm("norm_grad", 4 * 8191, 24, 8, 128, 64, True, True, True, 1 << 20),
        # the smallest call: a few tokens of a small model, weights in 32 bits
        _norm("norm_few", 3, 8, 2, 64, 64, False, False, True, 4096),
        # the gradient of a short, odd batch
        _norm("norm_grad_short", 517, 5, 1, 64, 32, False, True, False, 8192),
        # one new token of each of 64 running sequences, slices of one projection
        _append("append_step", 64, 1, 32768, 32, 8, 128, 128, False, 64, 512, True, 0, 3),
        # prompts of several requests written in chunks
        _append("append_chunk", 4, 8192, 32768, 32, 8, 128, 128, False, 64, 512, True, 0, 7),
        # one token of one short sequence, rotated only, at positions of the caller's
        _append("append_one", 1, 1, 1000, 8, 2, 64, 32, True, 16, 64, False, 77, 0),
        # a decode step of 64 forks of a 32K prompt, grouped heads
        _shared("shared_step", 1, 64, 1, 32768, 512, 32, 8, 128, 64, 2),
        # the smallest call: four answers to one short prompt
        _shared("shared_small", 1, 4, 1, 1024, 64, 8, 2, 64, 16, 0),
        # a kv head for each query head, answers already long
        _shared("shared_heads", 1, 16, 1, 16384, 2000, 32, 32, 128, 64, 5),
        # three prompts with several forks each, a few new tokens at once, five q heads to a kv head
        _shared("shared_groups", 3, 11, 5, 9000, 700, 20, 4, 64, 32, 9),
        # questions of up to 200 tokens on one long document
        _shared("shared_chunk", 1, 8, 200, 16384, 600, 32, 8, 128, 64, 4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "append", "shared", "shared", "shared"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
    rot = rng.choice([d, d, d // 2, 16])
    inter = rng.random() < 0.5
    if op == "norm":
        hq, hkv = rng.choice([(hq, hkv), (32, 8), (32, 32)])
        grad = rng.random() < 0.5
        most = 32768 * 64 * 128 // ((hq + hkv) * d)
        return {"op": "norm", "tokens": _log(rng, 1, min(most * 2 // 3 if grad else most, 100000)), "hq": hq, "hkv": hkv, "d": d,
                "rot": rot, "interleaved": inter, "grad": grad, "wide": rng.random() < 0.5, "far": _log(rng, 1000, 1 << 20)}
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        block = rng.choice([b for b in (64, 128, 256, 512, 1024, 2048) if b >= page])
        seqs = _log(rng, 1, 48)
        new = rng.choice([1, 1, _log(rng, 2, 8192)])
        new = max(1, min(new, 32768 // seqs))
        ctx = max(new, _log(rng, max(64, new), max(64, min(65536, (1 << 20) // seqs))))
        return {"op": "append", "seqs": seqs, "new": new, "ctx": ctx, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
                "interleaved": inter, "page": page, "block": block, "norm": rng.random() < 0.7,
                "shift": rng.choice([0, 0, _log(rng, 1, 1 << 20)]), "mix": rng.randrange(1, 1000)}
    groups = rng.choice([1, 1, 1, 2, 3, 5])
    seqs = _log(rng, 1, max(1, 96 // groups))
    new = rng.choice([1, 1, 1, _log(rng, 2, 16), _log(rng, 16, 300)])
    cells = (1 << 29) // (groups * seqs * hq)
    new = max(1, min(new, cells // 2048))
    tail = max(new, _log(rng, max(16, new), max(16, new, min(4096, (1 << 27) // (groups * seqs * hkv * d)))))
    most = min(65536, cells // new - tail, (1 << 27) // (groups * hkv * d))
    return {"op": "shared", "groups": groups, "seqs": seqs, "new": new, "prefix": _log(rng, 64, max(64, most)), "tail": tail,
            "hq": hq, "hkv": hkv, "d": d, "page": page, "mix": rng.randrange(0, 1000)}


def _lengths(case):
    """(new tokens, cache length with them) of each appended sequence: even for mix 0, else spread below the first one's."""
    n, new, ctx = case["seqs"], case["new"], case["ctx"]
    if case["mix"] == 0:
        return [new] * n, [ctx] * n
    r = random.Random(case["mix"])
    nq, lens = [new], [ctx]
    for _ in range(n - 1):
        length = r.randint(max(1, ctx // 8), ctx)
        lens.append(length)
        nq.append(0 if new > 1 and r.random() < 0.1 else min(length, r.randint((new + 7) // 8, new)))
    return nq, lens


def _forks(case):
    """Of each group its shared tokens (whole pages), and of its sequences the new tokens and the tokens behind the
    shared ones, new ones among them: even for mix 0, else spread below the first one's."""
    r = random.Random(case["mix"])
    out = []
    for g in range(case["groups"]):
        prefix = case["prefix"] if g == 0 or case["mix"] == 0 else r.randint(max(1, case["prefix"] // 4), case["prefix"])
        members = []
        for i in range(case["seqs"]):
            if (g == 0 and i == 0) or case["mix"] == 0:
                members.append((case["new"], case["tail"]))
            else:
                n = r.randint((case["new"] + 7) // 8, case["new"])
                members.append((n, r.randint(n, max(n, case["tail"]))))
        out.append((prefix // case["page"] * case["page"], members))
    return out


def _frequencies(rot):
    """Radians a position for each pair, in 64 bits, base 10000."""
    return 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=g.device, dtype=torch.bfloat16)


def _weight(g, d, wide):
    w = 1 + 0.25 * torch.randn(d, generator=g, device=g.device)
    return w if wide else w.bfloat16()


def _pages(case, g, lists, blocks_of):
    """Pools with shuffled pages, the page table (-1 where a sequence has no page) of ``lists`` (page numbers from 0
    up, in the order of the tokens), whose keys share an offset for each of ``blocks_of``."""
    page, hkv, d = case["page"], case["hkv"], case["d"]
    dev = g.device
    total = 1 + max(max(x) for x in lists)
    pages = total + 5
    order = torch.randperm(pages, generator=g, device=dev)[:total]
    table = torch.full((len(lists), max(len(x) for x in lists)), -1, dtype=torch.int32, device=dev)
    seq = torch.from_numpy(np.repeat(np.arange(len(lists)), [len(x) for x in lists])).to(dev)
    col = torch.from_numpy(np.concatenate([np.arange(len(x)) for x in lists])).to(dev)
    table[seq, col] = order[torch.from_numpy(np.concatenate([np.array(x) for x in lists])).to(dev)].to(torch.int32)
    k, v = _normal(g, pages, hkv, page, d), _normal(g, pages, hkv, page, d)
    blocks = torch.from_numpy(blocks_of).to(dev)
    offset = 0.5 * _normal(g, int(blocks.max()) + 1, hkv, d)
    k[order] = k[order] + offset[blocks][:, :, None, :]
    return k, v, table


def _sizes(nq, lens, dev):
    cu = np.concatenate([[0], np.cumsum(nq)])
    return {"cu_host": cu, "lens_host": np.array(lens), "cu": torch.from_numpy(cu).to(dev, torch.int32),
            "lens": torch.tensor(lens, dtype=torch.int32, device=dev)}


def _prepare_norm(s, case, g):
    t, dev = case["tokens"], g.device
    # slices of one projection, as a layer has them
    x = _normal(g, t, case["hq"] + 2 * case["hkv"], case["d"])
    s["q"], s["k"] = x[:, :case["hq"]], x[:, case["hq"]:case["hq"] + case["hkv"]]
    if case["grad"]:
        s["dq"], s["dk"] = _normal(g, t, case["hq"], case["d"]), _normal(g, t, case["hkv"], case["d"])
    first = torch.randint(0, max(1, case["far"] - t), (1,), generator=g, device=dev)
    s["positions"] = ((torch.arange(t, device=dev) + first) % case["far"]).to(torch.int32)


def _prepare_append(s, case, g):
    nq, lens = _lengths(case)
    page, block, dev = case["page"], case["block"], g.device
    counts = [-(-x // page) for x in lens]
    starts = np.concatenate([[0], np.cumsum(counts)])
    first = np.concatenate([[0], np.cumsum([-(-x // block) for x in lens])])
    of_page = np.concatenate([f + np.arange(c) * page // block for f, c in zip(first, counts)])
    s.update(_sizes(nq, lens, dev))
    s["k_pages"], s["v_pages"], table = _pages(case, g, [np.arange(a, b) for a, b in zip(starts[:-1], starts[1:])], of_page)
    width = -(-max(lens) // block) * (block // page)
    s["table"] = torch.full((len(lens), width), -1, dtype=torch.int32, device=dev)
    s["table"][:, :table.shape[1]] = table
    # pooled keys of the blocks that are complete before the call
    s["kbar_pages"] = torch.zeros(s["k_pages"].shape[0], case["hkv"], case["d"], device=dev)
    per = block // page
    full = [(x - n) // block * per for n, x in zip(nq, lens)]
    if sum(full):
        of = torch.cat([s["table"][b, :f] for b, f in enumerate(full)]).long()
        sums = s["k_pages"][of].sum(2, dtype=torch.float64).view(-1, per, case["hkv"], case["d"]).sum(1)
        s["kbar_pages"][of[per - 1::per]] = (sums / block).float()
    hq, hkv = case["hq"], case["hkv"]
    x = _normal(g, sum(nq), hq + 2 * hkv, case["d"])
    s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    s["positions"] = None
    if case["shift"]:
        _, pos = _rows(s)
        s["positions"] = (pos + case["shift"]).to(torch.int32)


def _prepare_shared(s, case, g):
    page, dev = case["page"], g.device
    lists, nq, lens, of_page, at, groups = [], [], [], [], 0, [0]
    prefixes = []
    for prefix, members in _forks(case):
        head = np.arange(at, at + prefix // page)
        at += len(head)
        of_page.append(len(of_page) + np.zeros(len(head), dtype=np.int64))
        prefixes.append(prefix)
        for n, tail in members:
            mine = np.arange(at, at + -(-tail // page))
            at += len(mine)
            of_page.append(len(of_page) + np.zeros(len(mine), dtype=np.int64))
            lists.append(np.concatenate([head, mine]))
            nq.append(n)
            lens.append(prefix + tail)
        groups.append(len(nq))
    s.update(_sizes(nq, lens, dev))
    s["k_pages"], s["v_pages"], s["table"] = _pages(case, g, lists, np.concatenate(of_page))
    s["groups_host"], s["prefix_host"] = groups, prefixes
    s["cu_groups"] = torch.tensor(groups, dtype=torch.int32, device=dev)
    s["prefix_lens"] = torch.tensor(prefixes, dtype=torch.int32, device=dev)
    s["q"] = _normal(g, sum(nq), case["hq"], case["d"])


def prepare(case, seed):
    g = torch.Generator(device=_dev()).manual_seed(seed)
    s = {"case": case}
    if case["op"] != "shared":
        s["freqs"] = torch.from_numpy(_frequencies(case["rot"])).to(g.device)
        wide = case.get("wide", False)
        s["wq"], s["wk"] = (_weight(g, case["d"], wide) for _ in range(2))
    {"norm": _prepare_norm, "append": _prepare_append, "shared": _prepare_shared}[case["op"]](s, case, g)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _angles(positions, freqs, grad=False):
    """cos and sin in 32 bits of angles in 64, [tokens][1][pairs]."""
    angle = positions.double()[:, None] * freqs
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    return c, -s if grad else s


def _turn(x, turns, interleaved):
    """Rotated x [T][H][D], 32 bits."""
    c, s = turns
    rot = 2 * c.shape[-1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = torch.stack((a * c - b * s, b * c + a * s), -1) if interleaved else torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y.flatten(-2) if interleaved else y, x[..., rot:]), -1)


def _scaled(x):
    """Rows of x over their root mean square, in 32 bits, and one over that root."""
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _plain_norm(s):
    c = s["case"]
    turns = _angles(s["positions"], s["freqs"], c["grad"])
    out = {}
    for n, w in (("q", s["wq"].float()), ("k", s["wk"].float())):
        y, r = _scaled(s[n])
        if not c["grad"]:
            out[n] = _turn(y * w, turns, c["interleaved"]).bfloat16()
            continue
        g = _turn(s["d" + n].float(), turns, c["interleaved"])
        out["dw" + n] = (g * y).sum((0, 1), dtype=torch.float64).float()
        g = g * w
        out["d" + n] = (r * (g - y * (g * y).mean(-1, keepdim=True))).bfloat16()
    return out


def _rows(s):
    """The sequence and position of each new token."""
    t = torch.arange(int(s["cu_host"][-1]), device=s["cu"].device)
    b = torch.bucketize(t, s["cu"][1:].long(), right=True)
    return b, t - s["cu"][b] + (s["lens"] - (s["cu"][1:] - s["cu"][:-1]))[b]


def _plain_append(s):
    c = s["case"]
    page, block = c["page"], c["block"]
    b, pos = _rows(s)
    turns = _angles(pos if s["positions"] is None else s["positions"], s["freqs"])
    q, k = (_scaled(s[n])[0] * w.float() if c["norm"] else s[n].float() for n, w in (("q", s["wq"]), ("k", s["wk"])))
    to, off = s["table"][b, pos // page].long(), pos % page
    s["k_pages"][to, :, off] = _turn(k, turns, c["interleaved"]).bfloat16()
    s["v_pages"][to, :, off] = s["v"]
    # the blocks that this call completes
    lens, nq = s["lens_host"], np.diff(s["cu_host"])
    before, after = (lens - nq) // block, lens // block
    done = after - before
    if done.sum():
        per = block // page
        seq = np.repeat(np.arange(len(lens)), done)
        col = np.repeat(before, done) + np.arange(done.sum()) - np.repeat(np.cumsum(done) - done, done)
        cols = torch.from_numpy(col[:, None] * per + np.arange(per)).to(b.device)
        of = s["table"][torch.from_numpy(seq).to(b.device)[:, None], cols].long()
        s["kbar_pages"][of[:, -1]] = (s["k_pages"][of].sum((1, 3), dtype=torch.float64) / block).float()
    return {"q": _turn(q, turns, c["interleaved"]).bfloat16(), **{n: s[n] for n in ("k_pages", "v_pages", "kbar_pages")}}


def _plain_shared(s):
    c = s["case"]
    page, hkv, d = c["page"], c["hkv"], c["d"]
    group = c["hq"] // hkv
    table = s["table"].clamp(min=0).long()
    dev = s["q"].device
    q = s["q"].float().view(-1, hkv, group, d) / math.sqrt(d)
    b_of, pos_of = _rows(s)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:-1], device=dev)

    def pages(pool, of):  # [..., pages] -> [..., kv heads][tokens][d], 32 bits
        return pool[of].transpose(-4, -3).flatten(-3, -2).float()

    for lo, hi, prefix in zip(s["groups_host"][:-1], s["groups_host"][1:], s["prefix_host"]):
        rows = slice(int(s["cu_host"][lo]), int(s["cu_host"][hi]))
        x = q[rows].permute(1, 2, 0, 3)  # [kv head][head of the group][row][d]
        n = x.shape[2]
        # the shared keys, once for all rows
        kp, vp = (pages(s[p], table[lo, :prefix // page]) for p in ("k_pages", "v_pages"))
        far = torch.matmul(x.reshape(hkv, -1, d), kp.transpose(-1, -2))
        # every sequence's own
        longest = int(s["lens_host"][lo:hi].max()) - prefix
        own_pages = table[lo:hi, prefix // page:prefix // page + -(-longest // page)]
        kt, vt = (pages(s[p], own_pages) for p in ("k_pages", "v_pages"))  # [seq][kv head][tokens][d]
        new = int(np.diff(s["cu_host"])[lo:hi].max())
        seq, pos = b_of[rows] - lo, pos_of[rows]
        j = torch.arange(rows.start, rows.stop, device=dev) - s["cu"][b_of[rows]]
        y = x.new_zeros(hi - lo, hkv, group, new, d)
        y[seq, :, :, j] = q[rows]
        near = torch.matmul(y, kt[:, :, None].transpose(-1, -2))[seq, :, :, j]  # [row][kv head][head][tokens]
        hidden = prefix + torch.arange(near.shape[-1], device=dev) > pos[:, None]
        near = near.masked_fill(hidden[:, None, None], -math.inf).permute(1, 2, 0, 3)
        far = far.view(hkv, group, n, prefix)
        top = near.amax(-1, keepdim=True)
        if prefix:
            top = torch.maximum(top, far.amax(-1, keepdim=True))
        far, near = far.sub_(top).exp_(), (near - top).exp()
        total = far.sum(-1, keepdim=True) + near.sum(-1, keepdim=True)
        w = y.new_zeros(hi - lo, hkv, group, new, near.shape[-1])
        w[seq, :, :, j] = near.permute(2, 0, 1, 3)
        o = torch.matmul(w, vt[:, :, None])[seq, :, :, j].permute(1, 2, 0, 3)
        o = (o + torch.matmul(far.flatten(1, 2), vp).view(hkv, group, n, d)) / total
        out[rows], lse[rows] = o.permute(2, 0, 1, 3), (top + total.log())[..., 0].permute(2, 0, 1)
    return {"out": out.view(-1, c["hq"], d).bfloat16(), "lse": lse.view(-1, c["hq"])}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own_norm(s):
    from long_context_sparse_moba_gb300 import ops
    c = s["case"]
    if c["grad"]:
        dq, dk, dwq, dwk = ops.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["freqs"],
                                                eps=EPS, interleaved=c["interleaved"])
        return {"dwq": dwq, "dq": dq, "dwk": dwk, "dk": dk}
    q, k = ops.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["freqs"], eps=EPS, interleaved=c["interleaved"])
    return {"q": q, "k": k}


def _own_append(s):
    from long_context_sparse_moba_gb300 import ops
    c = s["case"]
    wq, wk = (s["wq"], s["wk"]) if c["norm"] else (None, None)
    q = ops.paged_append_rope(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["kbar_pages"], s["table"], s["cu"], s["lens"],
                              c["new"], c["block"], s["freqs"], positions=s["positions"], q_weight=wq, k_weight=wk, eps=EPS,
                              interleaved=c["interleaved"])
    return {"q": q, **{n: s[n] for n in ("k_pages", "v_pages", "kbar_pages")}}


def _own_shared(s):
    from long_context_sparse_moba_gb300 import ops
    out, lse = ops.paged_attn_shared(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["lens"], s["case"]["new"],
                                     s["cu_groups"], s["prefix_lens"])
    return {"out": out, "lse": lse}


def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm": _own_norm, "append": _own_append, "shared": _own_shared}[op](s)
    return {"norm": _plain_norm, "append": _plain_append, "shared": _plain_shared}[op](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["op"] == "norm":
        values = case["tokens"] * (hq + hkv) * d
        weights = 2 * d * (4 if case["wide"] else 2) + (8 * d if case["grad"] else 0)
        each = 4 + 3 * case["rot"] / d
        return {"bytes": (6 if case["grad"] else 4) * values + 4 * case["tokens"] + weights,
                "flops": values * (2 * each if case["grad"] else each)}
    nbytes = flops = 0.0
    if case["op"] == "append":
        block = case["block"]
        nq, lens = _lengths(case)
        for n, length in zip(nq, lens):
            nbytes += 4 * n * d * (hq + 2 * hkv) + 4 * n / case["page"] + (4 * n if case["shift"] else 0)
            flops += n * (hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))
            done = length // block - (length - n) // block
            if done:  # keys of the first completed block that were there before, and the pooled keys
                nbytes += hkv * d * (2 * ((length - n) % block) + 4 * done)
                flops += hkv * d * done * block
        return {"bytes": nbytes, "flops": flops}
    for prefix, members in _forks(case):
        nbytes += 4.0 * prefix * hkv * d
        for n, tail in members:
            nbytes += 4.0 * tail * hkv * d + n * hq * (4 * d + 4)
            flops += 4.0 * d * hq * (n * (prefix + tail - n) + n * (n + 1) / 2)
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_turn(x, positions, freqs, interleaved, sign):
    """The pairs as complex numbers, multiplied by exp(+-i angle)."""
    pairs = freqs.numel()
    y = x.clone()
    place = torch.arange(pairs, device=x.device)
    re, im = (2 * place, 2 * place + 1) if interleaved else (place, place + pairs)
    angle = torch.outer(positions.double(), freqs) * sign
    z = torch.complex(y[..., re], y[..., im]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_norm(s):
    c, got = s["case"], {}
    for n in ("q", "k"):
        x, w = s[n].double(), s["w" + n].double()
        size = torch.linalg.vecdot(x, x)[..., None] / c["d"] + EPS
        if not c["grad"]:
            got[n] = _exact_turn(x * w / size.sqrt(), s["positions"], s["freqs"], c["interleaved"], 1.0)
            continue
        g = _exact_turn(s["d" + n].double(), s["positions"], s["freqs"], c["interleaved"], -1.0)
        got["dw" + n] = (g * x / size.sqrt()).sum(1).sum(0)
        along = torch.linalg.vecdot(g * w, x)[..., None]
        got["d" + n] = g * w / size.sqrt() - x * along / (c["d"] * size ** 1.5)
    return got


def _exact_append(s):
    c = s["case"]
    page, block = c["page"], c["block"]
    kp, vp, kb = s["k_pages"].double(), s["v_pages"].double(), s["kbar_pages"].double()
    stored, table, q = kp.clone(), s["table"].long(), []
    for b, (lo, hi, length) in enumerate(zip(s["cu_host"][:-1], s["cu_host"][1:], s["lens_host"])):
        lo, hi, length = int(lo), int(hi), int(length)
        p = torch.arange(length - (hi - lo), length, device=kp.device)
        turned = []
        for n in ("q", "k"):
            x = s[n][lo:hi].double()
            if c["norm"]:
                x = x * s["w" + n].double() / (torch.linalg.vecdot(x, x)[..., None] / c["d"] + EPS).sqrt()
            turned.append(_exact_turn(x, p + c["shift"], s["freqs"], c["interleaved"], 1.0))
        q.append(turned[0])
        kp[table[b, p // page], :, p % page] = turned[1]
        stored[table[b, p // page], :, p % page] = turned[1].bfloat16().double()
        vp[table[b, p // page], :, p % page] = s["v"][lo:hi].double()
        for blk in range((length - (hi - lo)) // block, length // block):
            of = table[b, blk * block // page:(blk + 1) * block // page]
            kb[of[-1]] = stored[of].mean((0, 2))  # of the keys as they are stored
    return {"q": torch.cat(q), "k_pages": kp, "v_pages": vp, "kbar_pages": kb}


def _exact_shared(s):
    """Every sequence by itself, over its own list of pages."""
    c = s["case"]
    hkv, d = c["hkv"], c["d"]
    q = s["q"].double().view(-1, hkv, c["hq"] // hkv, d)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:-1], dtype=torch.float64, device=q.device)
    for b, (lo, hi, length) in enumerate(zip(s["cu_host"][:-1], s["cu_host"][1:], s["lens_host"])):
        lo, hi, length = int(lo), int(hi), int(length)
        of = s["table"][b, :-(-length // c["page"])].long()
        at = (torch.arange(lo, hi, device=q.device) + length - hi)[:, None, None]
        for h in range(hkv):
            keys = s["k_pages"][of, h].reshape(-1, d)[:length].double()
            values = s["v_pages"][of, h].reshape(-1, d)[:length].double()
            logit = (q[lo:hi, h] @ keys.T * d ** -0.5).masked_fill(torch.arange(length, device=q.device) > at, -math.inf)
            z = torch.logsumexp(logit, -1)
            lse[lo:hi, h] = z
            out[lo:hi, h] = torch.exp(logit - z[..., None]) @ values
    return {"out": out.view(-1, c["hq"], d), "lse": lse.view(-1, c["hq"])}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "shared": _exact_shared}[case["op"]](s)
