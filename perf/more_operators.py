"""What is measured of the operators that carry a round's outcome on: the hypotheses that a beam keeps, and the states
that follow them.

  beams    the best continuations over a group's beams and the vocabulary
  reorder  the states of the beams (token counts, a cache) put in the order of what was kept
  write    keys and values of the rows that a round kept, rounded to 8 bits with a scale per 32 of them, into a cache
  read     the cache's entries read back

Formulas:
  beams    the candidate (r, v) of a group's row r has the score s_r + z_{r,v} - ln sum_v exp(z_{r,v}); a row that has ended has the one
           candidate (r, end_token) with the score s_r; rows with s_r = -inf and tokens with z = -inf have none.
           The n best in the order score descending, then row, then token.
  reorder  state[slot of i] <- what state[slot of rows[i]] held, as many positions as that slot's length says
  write    for 32 elements x of a head: e = the least integer >= -127 with max |x| <= 448 2^e; held are e + 127 and x 2^-e
           rounded to e4m3 (to nearest, ties to even)
  read     e4m3 value * 2^e, rounded once to the output's type
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# a full tree of 3, 2 and 1 children per depth: 16 nodes, the framework's measured tree
TREE = [-1, 0, 0, 0, 1, 1, 2, 2, 3, 3, 4, 5, 6, 7, 8, 9]
END = 2


def listed():
    c = dict(L=32, H=8, D=128, dtype="bf16")
    return [
        # one prompt, four beams of a small fp32 model: latency between two decode steps
        dict(op="beams", name="beams_b1_w4_v32000_fp32", dtype="fp32", B=1, W=4, V=32000, n=8, ended=0.0, first=False, masked=0.0),
        # an ordinary batch of eight beams each, a tenth of them ended; twice as many candidates as beams, so that W go on
        dict(op="beams", name="beams_b64_w8_v128256", dtype="bf16", B=64, W=8, V=128256, n=16, ended=0.1, first=False, masked=0.0),
        # the largest: wide beams over a large vocabulary, a quarter of the rows under a grammar
        dict(op="beams", name="beams_b128_w16_v152064", dtype="bf16", B=128, W=16, V=152064, n=32, ended=0.05, first=False, masked=0.25),
        # the token counts and bit arrays that the penalties read, of 64 groups of four beams
        dict(op="reorder", name="reorder_counts_b64_w4_v128256", kind="counts", B=64, W=4, V=128256),
        # one group's short cache: the launch counts
        dict(op="reorder", name="reorder_b1_w4_t512", kind="cache", B=1, W=4, L=4, T=512, H=8, D=128, shortest=300),
        # eight groups' 8-bit caches of ragged lengths, all layers of a model
        dict(op="reorder", name="reorder_b8_w8_t2048", kind="cache", B=8, W=8, L=16, T=2048, H=8, D=128, shortest=100),
        # one sequence's round, one layer: what its verify accepted of five rows
        dict(c, op="write", name="write_b1_k4_l1", rows="target", B=1, kmin=4, kmax=4, L=1, T=16, paged=True, held=1000),
        # a verify batch's accepted rows, all layers at once, into pages of 16 tokens
        dict(c, op="write", name="write_b64_k5_l32", rows="target", B=64, kmin=5, kmax=5, T=16, paged=True, held=500),
        # the accepted paths of candidate trees, fp32 keys, a head that ends inside a block of 32
        dict(c, op="write", name="write_tree_b32_n16_d80_fp32", dtype="fp32", rows="tree", B=32, kmin=15, kmax=15, L=8, H=5, D=80, T=512, paged=False, held=400),
        # eight prompts of ragged lengths, the cache filled for the first time
        dict(c, op="write", name="write_prompt_b8_t2048", rows="prompt", B=8, kmin=700, kmax=2048, L=16, T=64, paged=True, held=0),
        # one short sequence read back, one layer
        dict(c, op="read", name="read_b1_t500_l1", B=1, kmin=500, kmax=500, L=1, T=16, paged=True),
        # long sequences read back for a forward pass in 16 bits
        dict(c, op="read", name="read_b16_t8192_l4", B=16, kmin=1000, kmax=8192, L=4, T=64, paged=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["beams", "beams", "reorder", "write", "write", "read"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "beams":
        step = 8 if dtype == "bf16" else 4  # the framework's rows are multiples of 16 bytes
        V = step * max(1, _log_uniform(rng, 1000, 152064) // step)
        W = rng.choice([1, 2, 3, 4, 5, 8, 10, 16, 31, 64])
        most = 2000 * 152064 // (V * W * (2 if dtype == "fp32" else 1))  # no dearer than the largest listed case
        return dict(op=op, dtype=dtype, B=_log_uniform(rng, 1, max(1, min(512, most))), W=W, V=V, n=min(128, rng.choice([W, 2 * W, 2 * W + 1])),
                    ended=rng.choice([0.0, 0.1, 0.5]), first=rng.random() < 0.2, masked=rng.choice([0.0, 0.0, 0.3]))
    if op == "reorder":
        W = rng.choice([2, 3, 4, 5, 8, 16, 40])
        if rng.random() < 0.4:
            V = 4 * max(1, _log_uniform(rng, 1000, 152064) // 4)
            return dict(op=op, kind="counts", B=_log_uniform(rng, 1, max(1, min(128, 300 * 128256 // (V * W)))), W=W, V=V)
        L, T, H, D = rng.choice([1, 2, 4, 16]), _log_uniform(rng, 16, 2048), rng.choice([1, 4, 5, 8]), rng.choice([64, 80, 128])
        most = 60 * 16 * 2048 * 1024 // (L * T * H * D * W)
        return dict(op=op, kind="cache", B=_log_uniform(rng, 1, max(1, min(64, most))), W=W, L=L, T=T, H=H, D=D, shortest=rng.randint(0, T))
    L, H, D = rng.choice([1, 2, 4, 16, 32]), rng.choice([1, 4, 5, 8, 16]), rng.choice([64, 80, 96, 128, 192, 256])
    token = L * H * D * (2 if dtype == "fp32" else 1)
    if op == "read":
        kmax = _log_uniform(rng, 1, 4000)
        most = 16 * 4000 * 4 * 1024 // (token * kmax)
        B = _log_uniform(rng, 1, max(1, min(256, most)))
        if B * kmax * token > 16 * 4000 * 4 * 1024:
            kmax = max(1, 16 * 4000 * 4 * 1024 // (B * token))
        return dict(op=op, dtype=dtype, B=B, kmin=rng.randint(0, kmax), kmax=kmax, L=L, H=H, D=D, T=rng.choice([16, 64, 100]), paged=True)
    rows = rng.choice(["target", "target", "tree", "next", "prompt"])
    kmin, kmax = {"tree": (len(TREE) - 1,) * 2, "next": (0, 0), "prompt": (1, 500)}.get(rows) or (rng.randint(0, 4), rng.randint(4, 14))
    paged = rng.random() < 0.7
    T = rng.choice([16, 32, 100]) if paged else 600
    most = 8000 * 16 * 1024 // (token * (kmax + 1))
    if not paged:
        most = min(most, 10 ** 9 // (L * H * D * T))
    return dict(op=op, dtype=dtype, rows=rows, B=_log_uniform(rng, 1, max(1, min(256, most))), kmin=kmin, kmax=kmax, L=L, H=H, D=D, T=T,
                paged=paged, held=rng.randint(0, 100))


def _fixed(case, k=0):
    """Numbers that are the case's own, whatever the seed."""
    return np.random.RandomState(case["B"] + 1000 * k)


def _lengths(case):
    """Rows of each sequence (write: drafted tokens; read: tokens held)."""
    return _fixed(case).randint(case["kmin"], case["kmax"] + 1, case["B"]).astype(np.int64)


def _accepted(case):
    """Accepted tokens of each sequence; -1: its verify reported a data error."""
    k = _lengths(case)
    if case["rows"] == "tree":
        k = np.full_like(k, 3)
    n = (_fixed(case, 1).rand(case["B"]) * (k + 1)).astype(np.int64)
    return np.where(_fixed(case, 2).rand(case["B"]) < 0.01, -1, n) if case["B"] > 1 else n


def _kept(case):
    """Rows that a write puts into the cache."""
    if case["rows"] == "prompt":
        return int(_lengths(case).sum())
    return case["B"] if case["rows"] == "next" else int((_accepted(case) + 1).sum())


def _parents(case):
    """Of a group of W beams, which one each goes on from: some stay, some are taken twice or more."""
    W = case["W"]
    return np.sort(np.minimum(_fixed(case, 3).randint(0, W, (case["B"], W)), _fixed(case, 4).randint(0, W, (case["B"], W))), 1)


def _held(case):
    """Cached tokens of each group's beams (all of one length), for reorder."""
    return _fixed(case, 5).randint(case["shortest"], case["T"] + 1, case["B"]).astype(np.int64)


def _offsets(per):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(per)]).astype(np.int32)).cuda()


def _blocks(D):
    return -(-D // 32)


def _pool(g, shape, e=0):
    """A cache's contents: normal values in e4m3, and exponents' bytes."""
    x = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for part in x.view(shape[0], -1):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(100).clamp_(-448, 448))
    return x, torch.randint(112 + e, 122 + e, (*shape[:-1], _blocks(shape[-1])), generator=g, device="cuda", dtype=torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, B = case["op"], case["B"]
    rand = lambda *n: torch.rand(*n, generator=g, device="cuda")  # noqa: E731
    perm = lambda n: torch.randperm(n, generator=g, device="cuda")  # noqa: E731
    if op == "beams":
        W, V, R = case["W"], case["V"], case["B"] * case["W"]
        s = dict(op=op, n=case["n"], offsets=_offsets([W] * B))
        # logit rows: Zipf over random ranks with noise, as the framework's synthetic workloads
        z = rand(R, V).mul_(V).floor_().log1p_().mul_(-1.1).add_(torch.randn(R, V, generator=g, device="cuda"))
        strict = perm(R)[: int(R * case["masked"])]
        if len(strict):
            z[strict] = z[strict].masked_fill_(rand(len(strict), V) > 0.01, -math.inf)  # a grammar that allows one token in a hundred
        s["logits"] = z.to(DTYPES[case["dtype"]])
        s["scores"] = torch.randn(R, generator=g, device="cuda").mul_(2).sub_(20)
        if case["first"]:  # the first step: one prompt's row, the other beams are empty
            s["scores"][torch.arange(R, device="cuda") % W > 0] = -math.inf
        s["ended"] = torch.zeros(R, dtype=torch.bool, device="cuda")
        s["ended"][perm(R)[: int(R * case["ended"])]] = True
        return s
    if op == "reorder":
        W, S = case["W"], case["B"] * case["W"] + 1
        s = dict(op=op, kind=case["kind"], offsets=_offsets([W] * B), slots=perm(S)[: B * W].to(torch.int32))
        # which beam of its group each goes on from: the case's own map, its beams renamed by the seed
        name = torch.argsort(rand(B, W), 1)
        rows = torch.empty(B, W, dtype=torch.int64, device="cuda")
        rows.scatter_(1, name, name.gather(1, torch.from_numpy(_parents(case)).cuda()))
        s["rows"] = (rows + W * torch.arange(B, device="cuda").unsqueeze(1)).flatten().to(torch.int32)
        if case["kind"] == "counts":
            V = case["V"]
            s["counts"] = torch.poisson(rand(S, V), generator=g).to(torch.int32)
            s["seen"] = torch.randint(-(1 << 31), 1 << 31, (S, 2, -(-V // 32)), generator=g, device="cuda").to(torch.int32)
            return s
        s["k"], s["k_scale"] = _pool(g, (case["L"], S, case["T"], case["H"], case["D"]))
        s["v"], s["v_scale"] = _pool(g, (case["L"], S, case["T"], case["H"], case["D"]))
        s["lengths"] = torch.zeros(S, dtype=torch.int32, device="cuda")
        s["lengths"][s["slots"].long()] = torch.from_numpy(_held(case)).cuda().repeat_interleave(W).to(torch.int32)
        return s
    L, H, D, T = case["L"], case["H"], case["D"], case["T"]
    n = _lengths(case)
    s = dict(op=op, T=T, dtype=DTYPES[case["dtype"]], S=B + 2)
    s["slots"] = perm(B + 2)[:B].to(torch.int32)
    if op == "write":
        s["rows"] = case["rows"]
        per = n + (1 if case["rows"] == "tree" else 0)
        R = {"target": int(n.sum()) + B, "next": B}.get(case["rows"], int(per.sum()))
        s["offsets"] = _offsets(per)
        room = case["held"] + int(n.max()) + 1
        held = torch.from_numpy(_fixed(case, 6).randint(0, case["held"] + 1, B)).cuda() if case["held"] else torch.zeros(B, dtype=torch.int64, device="cuda")
        channels = torch.randn(2, H, D, generator=g, device="cuda").mul_(0.7).exp_()  # some channels are larger than others
        for name, c in zip(("keys", "values"), channels):
            s[name] = torch.empty(L, R, H, D, dtype=s["dtype"], device="cuda")
            for part in s[name]:
                part.copy_(torch.randn(R, H, D, generator=g, device="cuda").mul_(c))
        if case["rows"] in ("target", "tree"):
            s["num_accepted"] = torch.from_numpy(_accepted(case).astype(np.int32)).cuda()
        if case["rows"] == "tree":
            base = torch.tensor(TREE, device="cuda").repeat(B, 1)
            at = s["offsets"][:-1].long().unsqueeze(1)
            s["parent"] = torch.where(base < 0, base, base + at).flatten().to(torch.int32)
            # where the walk ended: one of the nodes of its depth
            depth = [[0], [1, 2, 3], [4, 5, 6, 7, 8, 9], [10, 11, 12, 13, 14, 15]]
            width = torch.tensor([1, 3, 6, 6], device="cuda")
            first = torch.tensor([d[0] for d in depth], device="cuda")
            d = s["num_accepted"].long().clamp(min=0)
            s["last_node"] = (at[:, 0] + first[d] + (rand(B) * width[d]).long()).to(torch.int32)
    else:
        room = int(n.max())
        held = torch.from_numpy(n).cuda()
        s["offsets"], s["R"] = _offsets(n), int(n.sum())
    s["lengths"] = torch.zeros(B + 2, dtype=torch.int32, device="cuda")
    s["lengths"][s["slots"].long()] = held.to(torch.int32)
    pages = B + 2
    if case["paged"]:
        each = -(-room // T)
        s["pages"] = perm((B + 2) * each).view(B + 2, each).to(torch.int32)
        pages = (B + 2) * each
    s["k"], s["k_scale"] = _pool(g, (L, pages, T, H, D))
    s["v"], s["v_scale"] = _pool(g, (L, pages, T, H, D), 2)
    if op == "write":
        s["out_lengths"] = torch.empty_like(s["lengths"])  # the next step's; a program keeps two and takes them in turn
    return s


def run(s):
    return {"beams": _beams, "reorder": _reorder, "write": _write, "read": _read}[s["op"]](s)


# ------------------------------------------------------------------- beams
def _beams(s):
    z, scores, n, ended = s["logits"], s["scores"], s["n"], s["ended"]
    if own:
        import speculative_decoding_verification_61_gb300 as sv
        return sv.spec_beam_select(z, scores, s["offsets"], n, ended=ended, end_token=END, lse=True)
    (R, V), B = z.shape, s["offsets"].numel() - 1
    live = (scores > -math.inf) & ~ended
    top = z.amax(1).double()
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    lse = (z.double() - top.unsqueeze(1)).exp_().sum(1).log() + top
    # each row's n best, and what ties with the last of them
    least = z.topk(min(n, V), 1).values[:, -1:]
    r, v = ((z >= least) & (z > -math.inf) & live.unsqueeze(1)).nonzero(as_tuple=True)
    score = scores.double()[r] + (z[r, v].double() - lse[r])
    done = (ended & (scores > -math.inf)).nonzero().squeeze(1)
    r, v, score = torch.cat([r, done]), torch.cat([v, torch.full_like(done, END)]), torch.cat([score, scores.double()[done]])
    group = torch.bucketize(r, s["offsets"][1:].long(), right=True)
    at = torch.argsort(r * V + v)
    at = at[torch.argsort(score[at], stable=True, descending=True)]
    at = at[torch.argsort(group[at], stable=True)]
    per = torch.bincount(group, minlength=B)
    rank = torch.arange(len(at), device=z.device) - (per.cumsum(0) - per)[group[at]]
    at, rank = at[rank < n], rank[rank < n]
    out_scores = torch.full((B, n), -math.inf, device=z.device)
    out_tokens = torch.full((B, n), -1, dtype=torch.int32, device=z.device)
    out_rows = out_tokens.clone()
    out_scores[group[at], rank] = score[at].float()
    out_tokens[group[at], rank] = v[at].to(torch.int32)
    out_rows[group[at], rank] = r[at].to(torch.int32)
    return out_scores, out_tokens, out_rows, torch.where(live, lse.float(), math.nan)


# ----------------------------------------------------------------- reorder
def _bytes(t):
    return t if t.dtype == torch.uint8 else t.view(torch.uint8)


def _reorder_plain(x, source, used=None):
    """x [.., S, ..] with the slots in dimension 0 of x, or 1 where positions (dimension 2) are used in part."""
    if used is None:
        return x.copy_(x[source])
    used = used.view(1, *used.shape, *[1] * (x.dim() - 3))
    return x.copy_(torch.where(used, x[:, source], x))


def _reorder(s):
    counts = s["kind"] == "counts"
    if own:
        import speculative_decoding_verification_61_gb300 as sv
        if counts:
            sv.spec_state_reorder([s["counts"], s["seen"]], s["rows"], s["offsets"], slots=s["slots"])
        else:
            sv.spec_state_reorder([(s[k], 1, 2) for k in ("k", "k_scale", "v", "v_scale")], s["rows"], s["offsets"], slots=s["slots"],
                                  lengths=s["lengths"])
    else:
        slots = s["slots"].long()
        source = torch.arange((s["counts"] if counts else s["lengths"]).shape[0], device=slots.device)
        source[slots] = slots[s["rows"].long()]
        if counts:
            _reorder_plain(s["counts"], source), _reorder_plain(s["seen"], source)
        else:
            used = torch.arange(s["k"].shape[2], device=slots.device) < s["lengths"][source].unsqueeze(1)
            _reorder_plain(_bytes(s["k"]), source, used), _reorder_plain(s["k_scale"], source, used)
            _reorder_plain(_bytes(s["v"]), source, used), _reorder_plain(s["v_scale"], source, used)
    if counts:
        return s["counts"], s["seen"]
    return s["k"], s["k_scale"].view(torch.float8_e8m0fnu), s["v"], s["v_scale"].view(torch.float8_e8m0fnu)


# ------------------------------------------------------------- write, read
def _in_blocks(x):
    """[.., D] -> [.., blocks, 32], the last block filled up with zeros."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % 32)).unflatten(-1, (-1, 32))


def _quantised(x):
    x32 = _in_blocks(x.float())
    m, e = torch.frexp(x32.abs().amax(-1))  # 0.5 <= m < 1: the largest is (2 m) 2^(e - 1), and 448 = 1.75 * 2^8
    e = torch.where(m > 0, e - 9 + (m > 0.875).to(e.dtype), torch.full_like(e, -127)).clamp_(min=-127)
    q = torch.ldexp(x32, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.flatten(-2)[..., : x.shape[-1]], (e + 127).to(torch.uint8)


def _place(s, slot, position):
    """The entry (page * T + place in it) of each position of a slot."""
    page = slot if s.get("pages") is None else s["pages"].long()[slot, position // s["T"]]
    return page * s["T"] + (position if s.get("pages") is None else position % s["T"])


def _write(s):
    names = ("k", "k_scale", "v", "v_scale")
    if own:
        import speculative_decoding_verification_61_gb300 as sv
        sv.spec_cache_write(*[s[k] for k in names], s["lengths"], s["keys"], s["values"], s["offsets"], rows=s["rows"], slots=s["slots"],
                            num_accepted=s.get("num_accepted"), parent=s.get("parent"), last_node=s.get("last_node"), pages=s.get("pages"),
                            out_lengths=s["out_lengths"])
    else:
        o, R, B = s["offsets"].long(), s["keys"].shape[1], s["slots"].numel()
        n, slots = s.get("num_accepted"), s["slots"].long()
        r, seq = torch.arange(R, device=o.device), torch.arange(B, device=o.device)
        first = o + torch.arange(B + 1, device=o.device) if s["rows"] == "target" else torch.arange(B + 1, device=o.device) if s["rows"] == "next" else o
        seq = torch.bucketize(r, first[1:], right=True)
        i = r - first[seq]  # which of its sequence's rows
        kept = torch.ones_like(r, dtype=torch.bool) if n is None else i <= n[seq]
        count = first.diff() if n is None else n.long() + 1
        if s["rows"] == "tree":
            nodes = len(TREE)
            up = torch.eye(nodes, device=o.device).repeat(B, 1, 1)
            local = s["parent"].long().view(B, nodes) - o[:-1].unsqueeze(1)
            up[:, torch.arange(1, nodes), :] += torch.nn.functional.one_hot(local[:, 1:], nodes).float()
            above = torch.matrix_power(up, 4) > 0  # of each node, itself and its ancestors
            path = above[torch.arange(B, device=o.device), s["last_node"].long() - o[:-1]] & (n >= 0).unsqueeze(1)
            kept, i = path.flatten(), (path.cumsum(1) - 1).flatten()
        r, seq, i = r[kept], seq[kept], i[kept]
        at = _place(s, slots[seq], s["lengths"].long()[slots[seq]] + i)
        for x, pool, scale in ((s["keys"], s["k"], s["k_scale"]), (s["values"], s["v"], s["v_scale"])):
            q, e = _quantised(x[:, r])
            _bytes(pool).flatten(1, 2)[:, at] = q
            scale.flatten(1, 2)[:, at] = e
        s["out_lengths"].copy_(s["lengths"])
        s["out_lengths"][slots] += count.to(torch.int32)
    return s["k"], s["k_scale"].view(torch.float8_e8m0fnu), s["v"], s["v_scale"].view(torch.float8_e8m0fnu), s["out_lengths"]


def _read(s):
    if own:
        import speculative_decoding_verification_61_gb300 as sv
        return sv.spec_cache_read(s["k"], s["k_scale"], s["v"], s["v_scale"], s["lengths"], s["offsets"], s["R"], slots=s["slots"], pages=s.get("pages"),
                                  dtype=s["dtype"])
    o = s["offsets"].long()
    r = torch.arange(s["R"], device=o.device)
    seq = torch.bucketize(r, o[1:], right=True)
    at = _place(s, s["slots"].long()[seq], r - o[seq])
    return tuple(_values(s[p].flatten(1, 2)[:, at], s[e].flatten(1, 2)[:, at]).to(s["dtype"]) for p, e in (("k", "k_scale"), ("v", "v_scale")))


def _values(q, e):
    x = _in_blocks(q.float())
    return torch.ldexp(x, (e.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)[..., : q.shape[-1]]


def work(case):
    op, B = case["op"], case["B"]
    if op == "beams":
        R, V = B * case["W"], case["V"]
        live = (B if case["first"] else R) * (1 - case["ended"])
        return {"bytes": live * V * (4 if case["dtype"] == "fp32" else 2) + R * 9 + B * case["n"] * 12, "flops": 4 * live * V}
    if op == "reorder":
        p = _parents(case)
        moved = p != np.arange(case["W"])
        read = np.array([len(set(row[m])) for row, m in zip(p, moved)])
        if case["kind"] == "counts":
            each = np.full(B, case["V"] * 4 + -(-case["V"] // 32) * 8)
        else:
            each = _held(case) * case["L"] * 2 * case["H"] * (case["D"] + _blocks(case["D"]))
        return {"bytes": float(((read + moved.sum(1)) * each).sum()) + B * case["W"] * 8, "flops": 0}
    size = 4 if case["dtype"] == "fp32" else 2
    tokens = _kept(case) if op == "write" else int(_lengths(case).sum())
    heads = tokens * case["L"] * 2 * case["H"]
    return {"bytes": heads * (case["D"] * (size + 1) + _blocks(case["D"])) + B * 16, "flops": heads * case["D"] * 2}


# ------------------------------------------------------- from the definitions, in 64 bits
def _e4m3(y):
    """The nearest multiple of the step that e4m3 has at y, ties to even."""
    _, e = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.round(y / step) * step


def _held_as(x):
    """A row of heads [H, D] of numbers: what e4m3 and the scales hold of it, and the scales."""
    H, D = x.shape
    q, scale = np.zeros((H, D)), np.zeros((H, _blocks(D)))
    for j in range(_blocks(D)):
        part = x[:, 32 * j: 32 * j + 32]
        big = np.abs(part).max(1)
        e = np.full(H, -127.0)
        np.maximum(np.ceil(np.log2(np.maximum(big, 1e-300) / 448)), -127, out=e)
        e = np.where(448 * 2.0 ** e < big, e + 1, np.where((e > -127) & (448 * 2.0 ** (e - 1) >= big), e - 1, e))
        q[:, 32 * j: 32 * j + 32] = _e4m3(part * 2.0 ** -e[:, None])
        scale[:, j] = 2.0 ** e
    return q, scale


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "beams":
        z, n, o = s["logits"], case["n"], s["offsets"].tolist()
        out, lse = torch.full((case["B"], n), -math.inf, dtype=torch.float64, device="cuda"), torch.full((z.shape[0],), math.nan, dtype=torch.float64, device="cuda")
        for b in range(case["B"]):
            found = []
            for r in range(o[b], o[b + 1]):
                score = float(s["scores"][r])
                if score == -math.inf:
                    continue
                if bool(s["ended"][r]):
                    found.append(torch.tensor([score], dtype=torch.float64, device="cuda"))
                    continue
                lse[r] = torch.logsumexp(z[r].double(), 0)
                p = z[r].double() - lse[r] + score
                found.append(p.sort(descending=True).values[:n])
            if found:
                best = torch.cat(found).sort(descending=True).values[:n]
                out[b, : len(best)] = best
        return out, None, None, lse
    if op == "reorder":
        return None  # values are moved, none is computed
    heads = (_kept(case) if op == "write" else s["R"]) * case["L"] * case["H"] * 2
    if heads * case["D"] > 30_000_000:
        return None
    first = s["offsets"].tolist()
    slots, held = s["slots"].tolist(), s["lengths"].tolist()
    pages = s["pages"].cpu().numpy() if case["paged"] else None
    T = case["T"]
    where = lambda slot, p: (slot, p) if pages is None else (pages[slot, p // T], p % T)  # noqa: E731
    if op == "read":
        outs = []
        for p, e in (("k", "k_scale"), ("v", "v_scale")):
            pool = s[p].double().cpu().numpy()
            scale = np.repeat(2.0 ** (s[e].double().cpu().numpy() - 127), 32, -1)[..., : case["D"]]
            out = np.zeros((case["L"], s["R"], case["H"], case["D"]))
            for b in range(case["B"]):
                for r in range(first[b], first[b + 1]):
                    at = where(slots[b], r - first[b])
                    out[:, r] = pool[:, at[0], at[1]] * scale[:, at[0], at[1]]
            outs.append(out)
        return tuple(outs)
    n = s["num_accepted"].tolist() if "num_accepted" in s else None
    outs, after = [], list(held)
    for x, p, e in ((s["keys"], "k", "k_scale"), (s["values"], "v", "v_scale")):
        x = x.double().cpu().numpy()
        pool, scale = s[p].double().cpu().numpy(), 2.0 ** (s[e].double().cpu().numpy() - 127)
        for b in range(case["B"]):
            if case["rows"] == "tree":
                path, node = [], int(s["last_node"][b]) if n[b] >= 0 else -1
                while node >= 0:
                    path.insert(0, node)
                    node = int(s["parent"][node])
            elif case["rows"] == "target":
                path = list(range(first[b] + b, first[b] + b + n[b] + 1))
            elif case["rows"] == "next":
                path = [b]
            else:
                path = list(range(first[b], first[b + 1]))
            for i, r in enumerate(path):
                at = where(slots[b], held[slots[b]] + i)
                for layer in range(case["L"]):
                    pool[layer][at], scale[layer][at] = _held_as(x[layer, r])
            after[slots[b]] = held[slots[b]] + len(path)
        outs += [pool, scale]
    return (*outs, np.array(after))
