"""The serving operators over a paged key/value cache, as measurable cases.

Three operators, reached through two entry points of the package:

* ``append``: a step's new keys and values, the keys rotated to their
  positions, into the pages of their sequences, and the rotated queries
  (``cp_cache_append``).
* ``paged``: the new tokens' attention over their sequences' pages
  (``cp_attn_paged`` without prefixes).
* ``prefix``: the same for a batch whose sequences share long prefixes, each
  held once in the cache and attended once for all of its sequences
  (``cp_attn_paged`` with prefixes).

Where ``own`` is false ``run`` computes the plain form: index arithmetic,
gathers, products, exp and sums in fp32 (angles in fp64), rounded once at the
end.  Where it is true it makes the package's calls.

A case's batch is ragged: its lengths come from the case's own ``ragged``
number, so that ``work`` can count them; its data come from the seed.
"""
import math
import random

import numpy as np
import torch

own = False


def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="bf16", Hq=32, Hkv=8, d=128, page=16, heads_first=False, causal=True,
             seqs=1, past=0, past_max=0, new=1, new_max=1, prefixes=0, prefix=0, pad=0, ragged=0,
             rope_dim=128, interleaved=False, base=500000.0, far=0)
    c.update(kw)
    return c


def listed():
    return [
        # One sequence, one token: the smallest step of an interactive user.
        _case("append_1", "append", past=1000, past_max=1000, ragged=1),
        # A full decode batch, a token each.
        _case("append_decode_200", "append", seqs=200, past=1, past_max=8192, page=32, ragged=2),
        # Prompts of one prefill step, 16K tokens of five sequences in all.
        _case("append_prompts_16k", "append", seqs=5, new=16384, new_max=16384, page=64, ragged=3),
        # Short drafts deep in long sequences: half the head rotated, pairs side by side, heads-first pages, padded batch.
        _case("append_drafts_d64", "append", dtype="fp16", Hq=16, Hkv=4, d=64, seqs=37, past=1, past_max=4000, new=1,
              new_max=9, rope_dim=32, interleaved=True, heads_first=True, base=10000.0, far=1000000, pad=7, ragged=4),
        # One sequence, one token, a short context: the latency of a single user's decode.
        _case("decode_1x1000", "paged", past=999, past_max=999, ragged=5),
        # The decode step of a busy server: 64 sequences of very different lengths in small pages.
        _case("decode_64_ragged", "paged", seqs=64, past=1, past_max=16384, ragged=6),
        # One sequence of a million tokens: the whole card works on one row of queries.
        _case("decode_1x1M", "paged", past=1048575, past_max=1048575, page=64, ragged=7),
        # Drafts of five tokens verified at once, small heads, heads-first pages, padded batch.
        _case("drafts_24x5_d64", "paged", dtype="fp16", Hq=16, Hkv=4, d=64, seqs=24, past=1, past_max=4093, new=5,
              new_max=5, heads_first=True, pad=8, ragged=8),
        # Chunks of prompts beside decoding sequences: long and short rows in one step.
        _case("chunk_2k_mixed", "paged", seqs=3, past=100, past_max=14000, new=1, new_max=2048, page=128, ragged=9),
        # A handful of users on a short system prompt that does not fill its last page.
        _case("prefix_7x2000", "prefix", seqs=7, past=1, past_max=300, prefixes=1, prefix=2000, ragged=10),
        # A decode batch on one long document.
        _case("prefix_64x32k", "prefix", seqs=64, past=1, past_max=1023, prefixes=1, prefix=32768, page=64, ragged=11),
        # A large batch on two long prompts of different lengths.
        _case("prefix_256x16k", "prefix", seqs=256, past=1, past_max=511, prefixes=2, prefix=16384, page=32, ragged=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "paged", "paged", "prefix", "prefix"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    c = _case("drawn", op, dtype=rng.choice(["bf16", "bf16", "fp16"]), Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 4, 7, 8]), d=d,
              page=rng.choice([16, 16, 32, 64, 128, 256]), heads_first=rng.random() < 0.3, ragged=rng.randrange(1 << 20),
              pad=rng.choice([0, 0, 0, 5]), rope_dim=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3,
              base=rng.choice([10000.0, 500000.0]))
    del c["name"]
    if op == "append":
        c["seqs"] = _log(rng, 1, 256)
        c["past_max"] = _log(rng, 1, 16384)
        c["new_max"] = _log(rng, 1, max(1, 16384 // c["seqs"]))
        c["far"] = rng.choice([0, 0, 100000, 1000000])
    elif op == "paged":
        c["new_max"] = rng.choice([1, 1, 1, 2, 4, 7, 33, 400])
        c["seqs"] = _log(rng, 1, 64 if c["new_max"] < 33 else 4)
        c["past_max"] = _log(rng, 1, 262144 // c["seqs"] if c["new_max"] < 33 else 8192)
        c["causal"] = rng.random() < 0.85
    else:
        c["seqs"] = _log(rng, 2, 128)
        c["past_max"] = _log(rng, 1, 600)
        c["prefixes"] = rng.choice([1, 1, 2, 3])
        c["prefix"] = _log(rng, 40, 1000000 // c["seqs"])
        c["new_max"] = rng.choice([1, 1, 1, 3])
    c["past"] = max(0, c["past_max"] // 50 - 1)
    return c


def lengths(case):
    """The batch's whole numbers, from the case alone: tokens already held and
    new ones of each sequence, and which sequences share which prefix."""
    r = random.Random(case["ragged"])
    B = case["seqs"]
    past = [r.randint(case["past"], case["past_max"]) for _ in range(B)]
    if case["new"] > 1 and case["new"] == case["new_max"] and case["op"] == "append":  # `new` tokens in all, in B parts
        cut = sorted(r.sample(range(1, case["new"]), B - 1))
        new = [b - a for a, b in zip([0] + cut, cut + [case["new"]])]
    else:
        new = [r.randint(case["new"], case["new_max"]) for _ in range(B)]
        new[0] = case["new_max"]
    if case["past"] != case["past_max"]:
        past[-1] = case["past_max"]
    P = case["prefixes"]
    first = [round(p * B / P) for p in range(P + 1)] if P else [0]
    plen = [max(1, case["prefix"] - (p * case["prefix"] * 7) // 16) for p in range(P)]
    of = [max([p for p in range(P) if first[p] <= b], default=-1) for b in range(B)]
    return dict(past=past, new=new, kv=[a + b for a, b in zip(past, new)], first=first, plen=plen, of=of, tokens=sum(new))


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    perm = random.Random(seed)
    n, ps, Hq, Hkv, d, t = lengths(case), case["page"], case["Hq"], case["Hkv"], case["d"], _dtype(case)
    B, P, N = case["seqs"], case["prefixes"], n["tokens"] + case["pad"]
    pages_of = [-(-k // ps) for k in n["kv"]]
    prefix_pages_of = [-(-k // ps) for k in n["plen"]]
    total = sum(pages_of) + sum(prefix_pages_of)
    pages = total + max(2, total // 16)
    ids = torch.from_numpy(np.random.RandomState(seed % (1 << 32)).permutation(pages).astype(np.int32))

    def table(counts, at):
        out = torch.zeros(len(counts), max(counts + [1]), dtype=torch.int32)
        for i, k in enumerate(counts):
            out[i, :k] = ids[at:at + k]
            at += k
        return out.cuda(), at

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32 if math.prod(shape) < 1 << 24 else t).to(t)

    page_table, at = table(pages_of, 0)
    prefix_table, _ = table(prefix_pages_of, at)
    shape = (pages, Hkv, ps, d) if case["heads_first"] else (pages, ps, Hkv, d)
    k_cache, v_cache = normal(*shape), normal(*shape)
    if case["heads_first"]:
        k_cache, v_cache = k_cache.transpose(1, 2), v_cache.transpose(1, 2)
    start = [0]
    for k in n["new"]:
        start.append(start[-1] + k)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(case=case, k_cache=k_cache, v_cache=v_cache, q_start=ints(start), kv_len=ints(n["kv"]), page_table=page_table,
             prefix_first=ints(n["first"]), prefix_len=ints(n["plen"]), prefix_table=prefix_table,
             keys_max=max(k + (n["plen"][p] if p >= 0 else 0) for k, p in zip(n["kv"], n["of"])), new_max=max(n["new"]),
             tokens=n["tokens"])
    # The projection writes query, key and value heads side by side.
    qkv = normal(N, (Hq + 2 * Hkv) * d).view(N, Hq + 2 * Hkv, d)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if case["op"] == "append":
        freqs = case["base"] ** (-np.arange(case["rope_dim"] // 2, dtype=np.float64) * 2 / case["rope_dim"])
        s["freqs"] = torch.from_numpy(freqs).cuda()
        s["q_out"] = torch.zeros(N, Hq, d, dtype=t, device="cuda")
        # Sequences that began elsewhere (a rank's share of a longer one): positions of their own.
        pos = [case["far"] + perm.randrange(1000) + a + i if case["far"] else a + i
               for a, b in zip(n["past"], n["new"]) for i in range(b)]
        s["positions"] = ints(pos + [0] * case["pad"])
    else:
        s["q"] = s["q"].contiguous()
        s["o"] = torch.zeros(N, Hq, d, dtype=t, device="cuda")
        s["lse"] = torch.zeros(Hq, N, dtype=torch.float32, device="cuda")
    if own:
        import context_long_sequence_gb300 as cpa
        s["cpa"] = cpa
        s["plan"] = cpa.PagedPlan(Hq, Hkv, d, page_size=ps, dtype=t, max_seqs=B, max_tokens=N, max_new=s["new_max"],
                                  max_pages=page_table.shape[1], max_prefixes=P, max_prefix_pages=prefix_table.shape[1] if P else 0,
                                  causal=case["causal"], rope_dim=case["rope_dim"] if case["op"] == "append" else 0,
                                  rope_base=case["base"], rope_interleaved=case["interleaved"])
        s["cache"] = cpa.PagedCache(k_cache, v_cache)
        s["batch"] = cpa.PagedBatch(s["q_start"], s["kv_len"], page_table, n_tokens=N,
                                    prefix_first=s["prefix_first"] if P else None, prefix_len=s["prefix_len"] if P else None,
                                    prefix_table=prefix_table if P else None, positions=s.get("positions"))
        if case["op"] != "append":
            s["workspace"] = cpa.alloc_paged_workspace(s["plan"])
    return s


def _of_tokens(s):
    """Sequence and place in it of every token that belongs to one."""
    t = torch.arange(s["tokens"], device="cuda")
    seq = torch.bucketize(t, s["q_start"][1:].long(), right=True)
    return t, seq, t - s["q_start"].long()[seq]


def _plain_append(s):
    c = s["case"]
    t, seq, i = _of_tokens(s)
    n = c["rope_dim"]
    angle = s["positions"].long()[t].double()[:, None] * s["freqs"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def rotated(x):
        x = x[t].float()
        a, b = (x[..., 0:n:2], x[..., 1:n:2]) if c["interleaved"] else (x[..., :n // 2], x[..., n // 2:n])
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([turned, x[..., n:]], -1).to(_dtype(c))

    at = s["kv_len"].long()[seq] - (s["q_start"][1:] - s["q_start"][:-1]).long()[seq] + i
    page = s["page_table"].long()[seq, at // c["page"]]
    s["q_out"][t] = rotated(s["q"])
    s["k_cache"][page, at % c["page"]] = rotated(s["k"])
    s["v_cache"][page, at % c["page"]] = s["v"][t]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_attention(s):
    c = s["case"]
    B, Hkv, ps = c["seqs"], c["Hkv"], c["page"]
    G = c["Hq"] // Hkv
    kv, new = s["kv_len"].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    j = torch.arange(s["keys_max"], device="cuda")[None]
    if c["prefixes"]:
        of = torch.bucketize(torch.arange(B, device="cuda"), s["prefix_first"][1:].long(), right=True)
        plen = s["prefix_len"].long()[of][:, None]
        mine = (j - plen).clamp(min=0)
        held = j < plen
        place = torch.where(held, j.expand(B, -1), mine)
        shared = s["prefix_table"].long()[of].gather(1, (place // ps).clamp(max=s["prefix_table"].shape[1] - 1))
        page = torch.where(held, shared, s["page_table"].long().gather(1, (mine // ps).clamp(max=s["page_table"].shape[1] - 1)))
    else:
        plen = torch.zeros_like(kv)[:, None]
        place = j.expand(B, -1)
        page = s["page_table"].long().gather(1, (place // ps).clamp(max=s["page_table"].shape[1] - 1))
    t, seq, i = _of_tokens(s)
    q = torch.zeros(B, s["new_max"], c["Hq"], c["d"], device="cuda")
    q[seq, i] = s["q"][t].float()
    q = q.view(B, s["new_max"], Hkv, G, c["d"]).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * s["new_max"], c["d"])
    key = s["k_cache"][page, place % ps].float().permute(0, 2, 3, 1)
    score = (torch.matmul(q, key) * c["d"] ** -0.5).view(B, Hkv, G, s["new_max"], -1)
    del key
    row = torch.arange(s["new_max"], device="cuda")
    last = (plen + kv[:, None] - new[:, None] + row + 1) if c["causal"] else (plen + kv[:, None]).expand(-1, s["new_max"])
    score = score.masked_fill((j[:, None] >= last[:, :, None])[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    del score
    total = p.sum(-1, keepdim=True)
    value = s["v_cache"][page, place % ps].float().permute(0, 2, 1, 3)
    out = torch.matmul(p.view(B, Hkv, G * s["new_max"], -1), value).view(B, Hkv, G, s["new_max"], c["d"]) / total.clamp(min=1e-30)
    lse = (top + torch.log(total))[..., 0]
    s["o"][t] = out.permute(0, 3, 1, 2, 4).reshape(B, s["new_max"], c["Hq"], c["d"])[seq, i].to(_dtype(c))
    s["lse"][:, t] = lse.permute(1, 2, 0, 3).reshape(c["Hq"], B, s["new_max"])[:, seq, i]
    return s["o"], s["lse"]


def run(state):
    s = state
    if own:
        cpa = s["cpa"]
        if s["case"]["op"] == "append":
            cpa.cp_cache_append(s["plan"], s["cache"], s["batch"], s["q"], s["k"], s["v"], s["q_out"])
            return s["q_out"], s["k_cache"], s["v_cache"]
        cpa.cp_attn_paged(s["plan"], s["cache"], s["batch"], s["q"], s["o"], s["lse"], s["workspace"])
        return s["o"], s["lse"]
    return _plain_append(s) if s["case"]["op"] == "append" else _plain_attention(s)


def work(case):
    n, Hq, Hkv, d = lengths(case), case["Hq"], case["Hkv"], case["d"]
    N = n["tokens"]
    if case["op"] == "append":
        # New q, k and v in, rotated q and the cache's new rows out; three operations a rotated value.
        return dict(bytes=2 * N * (Hq + 2 * Hkv) * d * 2 + 4 * N, flops=3 * N * (Hq + Hkv) * case["rope_dim"])
    keys = sum(n["kv"]) + sum(n["plen"])
    pairs = 0
    for past, new, p in zip(n["past"], n["new"], n["of"]):
        before = past + (n["plen"][p] if p >= 0 else 0)
        pairs += new * before + (new * (new + 1) // 2 if case["causal"] else new * new)
    return dict(bytes=2 * keys * Hkv * d * 2 + 2 * N * Hq * d * 2 + 4 * N * Hq + 4 * keys // case["page"], flops=4 * d * Hq * pairs)


def exact(case, seed):
    s, n, ps = prepare(case, seed), lengths(case), case["page"]
    half = case["rope_dim"] // 2
    a = 0
    if case["op"] == "append":
        q_out, kc, vc = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
        x, y = (np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)) if case["interleaved"] else (np.arange(half), np.arange(half, 2 * half))
        x, y = torch.from_numpy(x).cuda(), torch.from_numpy(y).cuda()
        rate = torch.exp(-math.log(case["base"]) * torch.arange(half, dtype=torch.float64, device="cuda") / half)
        for b in range(case["seqs"]):
            e = a + n["new"][b]
            place = torch.arange(n["past"][b], n["kv"][b], device="cuda")
            unit = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.outer(s["positions"][a:e].double(), rate))[:, None]
            turned = []
            for z in (s["q"][a:e].double(), s["k"][a:e].double()):
                w = torch.complex(z[..., x], z[..., y]) * unit
                z[..., x], z[..., y] = w.real, w.imag
                turned.append(z)
            q_out[a:e] = turned[0]
            pages = s["page_table"][b].long()[place // ps]
            kc[pages, place % ps] = turned[1]
            vc[pages, place % ps] = s["v"][a:e].double()
            a = e
        return q_out, kc, vc
    o, lse = s["o"].double(), s["lse"].double()
    G = case["Hq"] // case["Hkv"]
    shared = {}

    def keys(ids, count):
        rows = ids.long()[:-(-count // ps)]
        return [c[rows].reshape(-1, case["Hkv"], case["d"])[:count].double().transpose(0, 1) for c in (s["k_cache"], s["v_cache"])]

    for b in range(case["seqs"]):
        e, p = a + n["new"][b], n["of"][b]
        if p >= 0 and p not in shared:
            shared = {p: keys(s["prefix_table"][p], n["plen"][p])}
        parts = ([shared[p]] if p >= 0 else []) + [keys(s["page_table"][b], n["kv"][b])]
        before = (n["plen"][p] if p >= 0 else 0) + n["past"][b]
        q = s["q"][a:e].double().view(e - a, case["Hkv"], G, case["d"])
        for h in range(case["Hkv"]):
            k, v = (torch.cat([x[i][h] for x in parts]) for i in (0, 1))
            score = q[:, h].reshape(-1, case["d"]) @ k.T / math.sqrt(case["d"])
            if case["causal"]:
                reach = before + torch.arange(e - a, device="cuda").repeat_interleave(G)
                score = score.where(torch.arange(k.shape[0], device="cuda") <= reach[:, None], -math.inf)
            whole = torch.logsumexp(score, -1)
            o[a:e, h * G:(h + 1) * G] = (torch.exp(score - whole[:, None]) @ v).view(e - a, G, case["d"])
            lse[h * G:(h + 1) * G, a:e] = whole.view(e - a, G).T
        a = e
    return o, lse
