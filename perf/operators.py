"""What is measured of the operators that shape logits before they are sampled or verified.

  process   penalties for repeated tokens, per-token biases and grammar masks on packed logit rows
  state     the token counts that the penalties read: a sequence's prompt set up, a round's tokens added
  truncate  top-k, top-p and min-p: tokens outside the kept set become -inf
  both      process, then truncate, in one call

Formulas, for row r of sequence b and token v, all in 32 bits unless said:
  c    = output_counts[slot_b, v] + how often v is among the drafted tokens that precede row r
  seen = c > 0 or v in the prompt of b
  y    = seen ? (z > 0 ? z / rho_b : z * rho_b) : z
  y    = (y - phi_b * c) - pi_b * [c > 0]
  y    = y + bias_b(v)
  y    = allowed_r(v) ? y : -inf, then rounded once to the logits' type
Truncation keeps a prefix of the order (z descending, then index ascending): the first k; of these the
tokens whose mass before them is < p * Z, in 64 bits, w = exp((z - zmax) / T), Z = the mass of the first k;
of these the ones with (z - zmax) / T >= ln(min_p).  Rows of greedy sequences (T = 0) stay as they are.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# a full tree of 3, 2 and 1 children per depth: 16 nodes, the framework's measured tree
TREE = [-1, 0, 0, 0, 1, 1, 2, 2, 3, 3, 4, 5, 6, 7, 8, 9]


def listed():
    c = dict(dtype="bf16", rows="target", tokens=2000, bias=32, grammar=0.0)
    return [
        # one sequence, one new token: every microsecond of it is latency between two decode steps
        dict(c, op="process", name="process_b1_k0_v128256", B=1, kmin=0, kmax=0, V=128256),
        # an ordinary verify batch; half of the sequences answer in a grammar
        dict(c, op="process", name="process_b64_k5_v128256", B=64, kmin=5, kmax=5, V=128256, grammar=0.5),
        # the largest batch, ragged draft lengths: a throughput server
        dict(c, op="process", name="process_b512_k1to10_v128256", B=512, kmin=1, kmax=10, V=128256, grammar=0.25),
        # candidate trees under a grammar: each node has a mask of its own
        dict(c, op="process", name="process_tree_b64_n16_v128256", rows="tree", B=64, kmin=15, kmax=15, V=128256,
             grammar=1.0),
        # plain decoding, penalties alone, written over the model's own logits
        dict(c, op="inplace", name="inplace_b256_k0_v152064", B=256, kmin=0, kmax=0, V=152064, bias=0),
        # after a round: the emitted tokens of every sequence are counted
        dict(c, op="update", name="update_b512_k1to10_v128256", B=512, kmin=1, kmax=10, V=128256),
        # 64 requests join a running batch of 512: their slots are cleared, their prompts marked
        dict(c, op="reset", name="reset_n64_s512_v128256", B=64, kmin=0, kmax=0, V=128256, tokens=4000),
        # one sequence, one row, sampled with top-p
        dict(c, op="truncate", name="truncate_b1_k0_v128256", B=1, kmin=0, kmax=0, V=128256, kinds="p"),
        # a small fp32 model's verify, top-k and top-p together
        dict(c, op="truncate", name="truncate_b8_k4_v32000_fp32", dtype="fp32", B=8, kmin=4, kmax=4, V=32000, kinds="kp"),
        # the largest batch, every user's own mix of settings
        dict(c, op="truncate", name="truncate_b512_k1to10_v128256", B=512, kmin=1, kmax=10, V=128256, kinds="mixed"),
        # the drafter's rows of a verify batch, everything set
        dict(c, op="both", name="both_draft_b64_k5_v128256", rows="draft", B=64, kmin=5, kmax=5, V=128256, kinds="kp"),
        # large vocabulary, half of the sequences greedy
        dict(c, op="both", name="both_b256_k8_v152064", B=256, kmin=8, kmax=8, V=152064, grammar=0.25, kinds="greedy"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["process", "process", "inplace", "update", "reset", "truncate", "truncate", "both", "both"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    step = 8 if dtype == "bf16" else 4  # the framework's rows are multiples of 16 bytes
    V = step * max(1, _log_uniform(rng, 1000, 152064) // step)
    rows = rng.choice(["target", "target", "draft", "next", "tree"]) if op in ("process", "truncate", "both") else "target"
    kmin = rng.randint(0, 4)
    kmax = kmin + rng.randint(0, 10)
    if rows == "tree":
        kmin = kmax = len(TREE) - 1
    most = 3300 * 128256 // (V * (kmax + 1) * (2 if dtype == "fp32" else 1))  # no dearer than the largest listed case
    B = _log_uniform(rng, 1, max(1, min(512, most)))
    if rows == "draft":
        kmin, kmax = max(1, kmin), max(1, kmax)
    return dict(op=op, dtype=dtype, rows=rows, B=B, kmin=kmin, kmax=kmax, V=V, tokens=_log_uniform(rng, 1, 8000),
                bias=rng.choice([0, 1, 7, 64]), grammar=rng.choice([0.0, 0.3, 1.0]), kinds=rng.choice(["p", "k", "kp", "m", "mixed", "greedy"]))


def _ks(case):
    """Draft lengths: the case's own, whatever the seed."""
    return np.random.RandomState(case["B"]).randint(case["kmin"], case["kmax"] + 1, case["B"]).astype(np.int64)


def _row_count(case):
    total = int(_ks(case).sum())
    return {"target": total + case["B"], "tree": total + case["B"], "draft": total, "next": case["B"]}[case["rows"]]


def _offsets(case):
    per = _ks(case) + (1 if case["rows"] == "tree" else 0)
    return np.concatenate([[0], np.cumsum(per)]).astype(np.int32)


def _pack(bits):
    """[.., V] of truth values -> int32 words [.., ceil(V / 32)], bit v % 32 of word v // 32."""
    V = bits.shape[-1]
    bits = torch.nn.functional.pad(bits, (0, -V % 32)).view(*bits.shape[:-1], -1, 32)
    words = (bits.to(torch.int64) << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _unpack(words, V):
    return ((words.unsqueeze(-1) >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1).flatten(-2)[..., :V].bool()


def _zipf_tokens(g, n, V):
    """Token ids as a vocabulary ordered by frequency gives them: P(v) about 1 / (v + 10)."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return (10 * ((V / 10 + 1) ** u - 1)).long().clamp_(0, V - 1).to(torch.int32)


def _choice(g, values, n, dtype=torch.float32):
    at = torch.randint(len(values), (n,), generator=g, device="cuda")
    return torch.tensor(values, dtype=dtype, device="cuda")[at]


def _seen_share(case, share):
    """How likely each token is to be among a sequence's (share * tokens) Zipf draws."""
    v = torch.arange(case["V"], dtype=torch.float64, device="cuda")
    return share * case["tokens"] / ((v + 10) * math.log(case["V"] / 10 + 1))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, B, V, rows = case["op"], case["B"], case["V"], case["rows"]
    R, offsets = _row_count(case), _offsets(case)
    s = dict(op=op, rows=rows, B=B, V=V, R=R, offsets=torch.from_numpy(offsets).cuda())
    S = B if op != "reset" else 8 * B
    if op != "truncate":
        # the slots' history: how often each token was emitted (Poisson around its Zipf rate) and the prompt's tokens
        length = torch.rand(S, 1, generator=g, device="cuda", dtype=torch.float64) * 0.9 + 0.1
        lam = (length * _seen_share(case, 0.5)).float()
        counts = torch.poisson(lam, generator=g).to(torch.int32)
        prompt = torch.rand(S, V, generator=g, device="cuda") < lam
        s["counts"], s["seen"] = counts, torch.stack([_pack(prompt), _pack(counts > 0)], 1).contiguous()
        s["slots"] = torch.randperm(S, generator=g, device="cuda")[:B].to(torch.int32)
    if op == "reset":
        n = torch.randint(0, case["tokens"] + 1, (B,), generator=g, device="cuda")
        m = torch.where(torch.rand(B, generator=g, device="cuda") < 0.25, n // 4, torch.zeros_like(n))  # resumed requests
        zero = torch.zeros(1, dtype=torch.int64, device="cuda")
        s["prompt_offsets"] = torch.cat([zero, n.cumsum(0)]).to(torch.int32)
        s["output_offsets"] = torch.cat([zero, m.cumsum(0)]).to(torch.int32)
        s["prompt_tokens"] = _zipf_tokens(g, int(n.sum()), V)
        s["output_tokens"] = _zipf_tokens(g, int(m.sum()), V)
        return s
    if op == "update":
        s["out_tokens"] = _zipf_tokens(g, R, V)
        k = s["offsets"].diff().float()
        n = (torch.rand(B, generator=g, device="cuda") * (k + 1)).to(torch.int32).minimum(k.to(torch.int32))
        bad = torch.rand(B, generator=g, device="cuda") < 0.01  # a sequence that the verify reported as a data error
        s["num_accepted"] = torch.where(bad, torch.full_like(n, -1), n)
        return s
    # logit rows: Zipf over random ranks with noise, as the framework's synthetic workloads
    z = torch.rand(R, V, generator=g, device="cuda").mul_(V).floor_().log1p_().mul_(-1.1)
    s["logits"] = z.add_(torch.randn(R, V, generator=g, device="cuda")).to(DTYPES[case["dtype"]])
    if op != "truncate":
        s["draft_tokens"] = _zipf_tokens(g, int(offsets[-1]), V)
        if rows == "tree":
            base = torch.tensor(TREE, device="cuda").repeat(B, 1)
            at = s["offsets"][:-1].long().unsqueeze(1)
            s["parent"] = torch.where(base < 0, base, base + at).flatten().to(torch.int32)
        s["repetition"] = _choice(g, [1.0, 1.05, 1.1, 1.3], B)
        s["frequency"] = _choice(g, [0.0, 0.1, 0.5], B)
        s["presence"] = _choice(g, [0.0, 0.2, 1.0], B)
        if case["bias"]:
            n = case["bias"]
            s["bias_offsets"] = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
            first = torch.randint(V, (B, 1), generator=g, device="cuda")
            gap = max(1, V // (n + 1))
            s["bias_tokens"] = ((first + gap * torch.arange(n, device="cuda")) % V).flatten().to(torch.int32)
            s["bias_values"] = _choice(g, [-100.0, -2.0, 1.5, 5.0], B * n)
        if case["grammar"]:
            # rows under a grammar: few tokens allowed (a key, a digit) or most of them (inside a string)
            seq = _row_seq(s)
            strict = torch.rand(B, generator=g, device="cuda") < case["grammar"]
            rule = strict[seq]
            M = max(1, int(rule.sum()))
            share = _choice(g, [0.0005, 0.01, 0.9], M).unsqueeze(1)
            s["mask"] = _pack(torch.rand(M, V, generator=g, device="cuda") < share)
            s["mask_rows"] = torch.where(rule, rule.long().cumsum(0) - 1, torch.full_like(seq, -1)).to(torch.int32)
    if op in ("truncate", "both"):
        kinds = case["kinds"]
        s["temperature"] = _choice(g, [0.7, 1.0, 1.0, 1.3], B)
        if kinds == "greedy":
            s["temperature"][1::2] = 0.0
        if kinds in ("k", "kp", "mixed", "greedy"):
            s["top_k"] = _choice(g, [0, 1, 20, 50, 1000] if kinds == "mixed" else [20, 50, 200], B, torch.int32)
        if kinds in ("p", "kp", "mixed", "greedy"):
            s["top_p"] = _choice(g, [0.5, 0.9, 0.95, 1.0] if kinds == "mixed" else [0.8, 0.9, 0.95], B)
        if kinds in ("m", "mixed"):
            s["min_p"] = _choice(g, [0.0, 0.02, 0.1], B)
    return s


PROCESS = ("repetition", "frequency", "presence", "counts", "seen", "slots", "bias_offsets", "bias_tokens", "bias_values", "mask", "mask_rows", "parent")
TRUNCATE = ("top_k", "top_p", "min_p")


def _given(s, names):
    return {n: s[n] for n in names if n in s}


def run(state):
    s = state
    if own:
        import speculative_decoding_verification_61_gb300 as sv

        if s["op"] in ("process", "inplace"):
            return sv.spec_logits_process(s["logits"], s["offsets"], s["draft_tokens"], rows=s["rows"],
                                          out=s["logits"] if s["op"] == "inplace" else None, **_given(s, PROCESS))
        if s["op"] == "truncate":
            return sv.spec_logits_truncate(s["logits"], s["temperature"], s["offsets"], rows=s["rows"], **_given(s, TRUNCATE))
        if s["op"] == "both":
            return sv.spec_logits_process_truncate(s["logits"], s["temperature"], s["offsets"], s["draft_tokens"], rows=s["rows"],
                                                   **_given(s, PROCESS), **_given(s, TRUNCATE))
        if s["op"] == "update":
            return sv.spec_penalty_update(s["counts"], s["seen"], s["out_tokens"], s["num_accepted"], s["offsets"], slots=s["slots"])
        return sv.spec_penalty_reset(s["counts"], s["seen"], s["slots"], s["prompt_offsets"], s["prompt_tokens"],
                                     s["output_offsets"], s["output_tokens"])
    if s["op"] == "process":
        return _process(s)
    if s["op"] == "inplace":
        return s["logits"].copy_(_process(s))
    if s["op"] == "truncate":
        return _truncate(s, s["logits"])
    if s["op"] == "both":
        return _truncate(s, _process(s))
    return _update(s) if s["op"] == "update" else _reset(s)


def _row_seq(s):
    """The sequence of each row."""
    per = {"target": s["offsets"].diff() + 1, "next": torch.ones_like(s["offsets"][1:])}.get(s["rows"], s["offsets"].diff())
    return torch.repeat_interleave(torch.arange(s["B"], device=per.device), per.long(), output_size=s["R"])


def _preceding(s, seq):
    """(row, token) of every drafted token that precedes a row."""
    row, off, d = torch.arange(s["R"], device=seq.device), s["offsets"].long(), s["draft_tokens"].long()
    if s["rows"] == "tree":  # the node's own token and its ancestors', the root's left out
        up = s["parent"].long()
        a1 = torch.where(up >= 0, up[up], up)
        a2 = torch.where(a1 >= 0, up[a1], a1)
        node = torch.stack([row, up, a1, a2], 1)
        ok = (node >= 0) & (up[node.clamp(min=0)] >= 0)
    else:
        first = {"target": off[:-1] + torch.arange(s["B"], device=seq.device), "draft": off[:-1]}.get(s["rows"])
        before = row - first[seq] if first is not None else off.diff()
        j = torch.arange(32, device=seq.device)
        node = off[:-1][seq].unsqueeze(1) + j
        ok = j < before.unsqueeze(1)
    return row.unsqueeze(1).expand_as(node)[ok], d[node[ok]]


def _process(s):
    V, z = s["V"], s["logits"].float()
    seq = _row_seq(s)
    slot = s["slots"].long()[seq]
    c = s["counts"][slot]
    row, token = _preceding(s, seq)
    c.view(-1).index_add_(0, row * V + token, torch.ones_like(token, dtype=torch.int32))
    seen = _unpack(s["seen"][:, 0], V)[slot] | (c > 0)
    rho, phi, pi = (s[n][seq].unsqueeze(1) for n in ("repetition", "frequency", "presence"))
    y = torch.where(seen, torch.where(z > 0, z / rho, z * rho), z)
    y = (y - phi * c.float()) - pi * (c > 0).float()
    if "bias_tokens" in s:
        n = s["bias_offsets"].diff().long()
        owner = torch.repeat_interleave(torch.arange(s["B"], device=z.device), n, output_size=s["bias_tokens"].numel())
        bias = torch.zeros(s["B"], V, device=z.device)
        bias.view(-1).index_add_(0, owner * V + s["bias_tokens"].long(), s["bias_values"])
        y = y + bias[seq]
    if "mask" in s:
        rule = s["mask_rows"].long()
        allowed = _unpack(s["mask"], V)[rule.clamp(min=0)] | (rule < 0).unsqueeze(1)
        y = torch.where(allowed, y, torch.full_like(y, -math.inf))
    return y.to(s["logits"].dtype)


def _truncate(s, logits):
    V, seq = s["V"], _row_seq(s)
    T = s["temperature"][seq].double().unsqueeze(1)
    z, at = logits.float().sort(dim=1, descending=True, stable=True)
    top = z[:, :1].double()
    x = (z.double() - top) / T
    w = x.exp()
    place = torch.arange(V, device=z.device)
    keep = torch.ones_like(z, dtype=torch.bool)
    if "top_k" in s:
        k = s["top_k"][seq].unsqueeze(1)
        keep &= (place < k) | (k == 0)
        w = w * keep
    if "top_p" in s:
        p = s["top_p"][seq].double().unsqueeze(1)
        mass = w.cumsum(1)
        keep &= (mass - w < p * mass[:, -1:]) | (p >= 1)
    if "min_p" in s:
        keep &= x >= s["min_p"][seq].double().unsqueeze(1).log()
    keep = torch.zeros_like(keep).scatter_(1, at, keep)
    same = (T == 0) | ~(top.abs() < math.inf)  # greedy rows, rows with NaN, +inf or nothing at all
    return torch.where(keep | same, logits, torch.full_like(logits, -math.inf))


def _update(s):
    counts, seen, V = s["counts"], s["seen"], s["V"]
    seq = _row_seq(s)
    first = s["offsets"][:-1].long() + torch.arange(s["B"], device=seq.device)
    emitted = torch.arange(s["R"], device=seq.device) - first[seq] <= s["num_accepted"][seq]
    slot, token = s["slots"].long()[seq][emitted], s["out_tokens"].long()[emitted]
    counts.view(-1).index_add_(0, slot * V + token, torch.ones_like(token, dtype=torch.int32))
    word = token // 32
    v = word.unsqueeze(1) * 32 + torch.arange(32, device=seq.device)
    there = (counts.view(-1)[(slot.unsqueeze(1) * V + v).clamp(max=counts.numel() - 1)] > 0) & (v < V)
    seen[slot, 1, word] = _pack(there).squeeze(1)
    return counts, seen


def _reset(s):
    counts, seen, V, n = s["counts"], s["seen"], s["V"], s["slots"].numel()
    dev, slots = counts.device, s["slots"].long()
    owner = torch.arange(n, device=dev)
    prompt = torch.zeros(n, V, dtype=torch.bool, device=dev)
    prompt[torch.repeat_interleave(owner, s["prompt_offsets"].diff().long(), output_size=s["prompt_tokens"].numel()), s["prompt_tokens"].long()] = True
    new = torch.zeros(n * V, dtype=torch.int32, device=dev)
    who = torch.repeat_interleave(owner, s["output_offsets"].diff().long(), output_size=s["output_tokens"].numel())
    new.index_add_(0, who * V + s["output_tokens"].long(), torch.ones_like(s["output_tokens"]))
    new = new.view(n, V)
    counts[slots] = new
    seen[slots] = torch.stack([_pack(prompt), _pack(new > 0)], 1)
    return counts, seen


def work(case):
    """Bytes that an operator has to read and write once each; sums and products are few beside them."""
    B, V, R, op = case["B"], case["V"], _row_count(case), case["op"]
    size, words = DTYPES[case["dtype"]].itemsize, -(-V // 32)
    v = np.arange(V)
    rate = 0.5 * case["tokens"] * 0.55 / ((v + 10) * math.log(V / 10 + 1))
    distinct = float((1 - np.exp(-rate)).sum())  # emitted tokens of one sequence; as many of its prompt
    if op == "update":
        n = 0.5 * (R + B)  # emitted tokens: half of the drafts and one more
        return {"bytes": 4 * R + 12 * B + 16 * n, "flops": 0}
    if op == "reset":
        n = case["tokens"] / 2 * (1 + 1 / 16) * B
        return {"bytes": B * (4 * V + 8 * words + 12) + 4 * n, "flops": 0}
    total, flops = 12.0 * B, 0.0
    if op in ("process", "inplace", "both"):
        total += B * (8 * words + 4 * distinct + 8 * case["bias"]) + 4 * R * case["grammar"] * words
        flops += R * 2 * distinct * 6
    if op == "inplace":
        # the tokens seen are read and written, and what a grammar takes away is written
        return {"bytes": total + 2 * size * R * 2 * distinct + 0.7 * size * R * V * case["grammar"], "flops": flops}
    if op in ("truncate", "both"):
        flops += 4.0 * R * V
    return {"bytes": total + 2 * size * R * V, "flops": flops}


def exact(case, seed):
    """From the definition in 64 bits: a formula for one token at a time, thresholds by bisection instead of a sort."""
    s = prepare(case, seed)
    if s["op"] in ("update", "reset"):
        return None  # whole numbers
    V, B, R = s["V"], s["B"], s["R"]
    off = s["offsets"].cpu().numpy().astype(np.int64)
    seq = np.empty(R, np.int64)
    before = []  # the drafted tokens that precede each row
    draft = s["draft_tokens"].cpu().numpy() if "draft_tokens" in s else None
    r = 0
    for b in range(B):
        n = int(off[b + 1] - off[b])
        for i in range({"target": n + 1, "next": 1}.get(s["rows"], n)):
            seq[r] = b
            if draft is not None and s["rows"] == "tree":
                path, node = [], i
                while node > 0:
                    path.append(draft[off[b] + node])
                    node = TREE[node]
                before.append(path)
            elif draft is not None:
                before.append(draft[off[b]:off[b] + (n if s["rows"] == "next" else i)])
            r += 1
    seq = torch.from_numpy(seq).cuda()
    z = s["logits"].double()
    if s["op"] != "truncate":
        for r0 in range(0, R, 256):
            z[r0:r0 + 256] = _exact_rows(s, z[r0:r0 + 256], seq[r0:r0 + 256], before[r0:r0 + 256], r0)
    if s["op"] in ("process", "inplace"):
        return z
    z = z.to(s["logits"].dtype).double()
    for r0 in range(0, R, 256):
        z[r0:r0 + 256] = _exact_kept(s, z[r0:r0 + 256], seq[r0:r0 + 256])
    return z


def _exact_rows(s, z, seq, before, r0):
    V, n = s["V"], z.shape[0]
    slot = s["slots"].long()[seq]
    drafted = torch.zeros(n, V, dtype=torch.float64, device=z.device)
    for i, path in enumerate(before):
        for t in path:
            drafted[i, int(t)] += 1
    c = s["counts"][slot].double() + drafted
    v = torch.arange(V, device=z.device)
    bit = lambda words: (words[:, v // 32] >> (v % 32).to(torch.int32)) & 1  # noqa: E731
    seen = (bit(s["seen"][slot, 0]) == 1) | (c > 0)
    rho, phi, pi = (s[k].double()[seq][:, None] for k in ("repetition", "frequency", "presence"))
    scale = torch.where(seen, torch.where(z > 0, 1 / rho, rho), torch.ones_like(z))
    y = z * scale - phi * c - pi * (c > 0)
    if "bias_tokens" in s:
        per = s["bias_tokens"].numel() // s["B"]
        for e in range(per):
            at = seq * per + e
            y[torch.arange(n, device=z.device), s["bias_tokens"][at].long()] += s["bias_values"][at].double()
    if "mask" in s:
        rule = s["mask_rows"][r0:r0 + n].long()
        y = torch.where((rule[:, None] >= 0) & (bit(s["mask"][rule.clamp(min=0)]) == 0), -math.inf, y)
    return y


def _exact_kept(s, z, seq):
    """z with -inf outside the kept set: the boundary value by bisection over the order of 32-bit floats, then its ties."""
    T = s["temperature"].double()[seq][:, None]
    top = z.max(1, keepdim=True).values
    w = ((z - top) / T).exp()
    key = z.float().view(torch.int32).long()
    key = torch.where(key < 0, -(key & 0x7FFFFFFF), key)

    def prefix(weight, most, on):
        """Tokens of the order (z descending, index ascending) whose weight before them is below `most`."""
        lo, hi = key.min(1, keepdim=True).values - 1, key.max(1, keepdim=True).values
        for _ in range(33):  # the lowest key with less than `most` above it
            mid = (lo + hi) // 2
            low = torch.where(key > mid, weight, 0.0).sum(1, keepdim=True) < most
            hi, lo = torch.where(low, mid, hi), torch.where(low, lo, mid)
        above = torch.where(key > hi, weight, 0.0).sum(1, keepdim=True)
        tie = key == hi
        rank = (tie.long().cumsum(1) - 1).double()
        return (key > hi) | (tie & (above + rank * weight < most)) | ~on

    keep = torch.ones_like(key, dtype=torch.bool)
    if "top_k" in s:
        k = s["top_k"].double()[seq][:, None]
        keep = prefix(torch.ones_like(z), k, k > 0)
    if "top_p" in s:
        p = s["top_p"].double()[seq][:, None]
        inside = torch.where(keep, w, 0.0)
        keep &= prefix(inside, p * inside.sum(1, keepdim=True), p < 1)
    if "min_p" in s:
        keep &= z >= top + T * s["min_p"].double()[seq][:, None].log()
    same = (T == 0) | ~top.isfinite()
    return torch.where(keep | same, z, -math.inf)
