"""Operators around the attention of a serving step, as measurable cases.

Four groups of cases:

* ``rope``: the rotation of whole sequences by positions of several axes (time,
  height, width), and its gradient (``cp_rope``).
* ``append``: a step's keys and values into their pages with such positions
  (``cp_cache_append`` with ``rope_axes``).
* ``verify``: drafted tokens against the target's probabilities, from given
  random numbers (``cp_verify_drafts``).
* ``pages``: the pages of the cache: what a step frees and takes
  (``cp_pages_resize``), sequences forked (``cp_pages_fork``), the cache made
  dense (``cp_pages_compact``), and the copies of the last two over the layers'
  caches (``cp_pages_copy``).

Where ``own`` is false ``run`` computes the plain form: index arithmetic,
gathers, scatters, products and sums in fp32 (angles and the sums that a random
number is compared with in fp64), rounded once at the end.  Where it is true
it makes the package's calls.

What decides how much work a case is (lengths, how many pages are held) comes
from the case's own ``ragged`` number, so that ``work`` can count it; the data
and which pages they are come from the seed.
"""
import math
import random

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- cases

def _rope(name, **kw):
    c = dict(name=name, op="rope", n=1024, Hq=32, Hkv=8, d=128, rope_dim=128, axes=3, cycled=False, interleaved=False,
             base=500000.0, dtype="bf16", inverse=False, out="same", far=0)
    c.update(kw)
    return c


def _append(name, **kw):
    c = dict(name=name, op="append", dtype="bf16", Hq=32, Hkv=8, d=128, page=16, heads_first=False, seqs=1, past=0, past_max=0,
             new=1, new_max=1, pad=0, ragged=0, rope_dim=128, axes=3, cycled=False, interleaved=False, base=500000.0, far=0)
    c.update(kw)
    return c


def _verify(name, **kw):
    c = dict(name=name, op="verify", seqs=1, drafts=4, drafts_max=4, vocab=128000, row=128000, dtype="fp32", drafter=True, rejected=1.0,
             pad=0, ragged=0)
    c.update(kw)
    return c


def _pages(name, what, **kw):
    c = dict(name=name, op="pages", what=what, rows=64, page=16, length=1000, new=5, replaced=0, parents=0, pages=8192, used=0.5,
             layers=1, Hkv=8, d=128, heads_first=False, dtype="bf16", ragged=0)
    c.update(kw)
    return c


def listed():
    return [
        # The queries and keys of one training sequence of text and images, a pair's axis by sections of the head.
        _rope("rope_train_64k", n=65536),
        # Their gradients as the attention's backward gives them (fp32), turned back and rounded for the projections' backward;
        # an odd length, an image tower's head, axes that take turns.
        _rope("rope_grad_5k_d80", n=5003, Hq=16, Hkv=16, d=80, rope_dim=80, axes=2, cycled=True, inverse=True, out="fp32_in", base=10000.0),
        # One sequence, one token: the smallest step of a user who talks about a picture.
        _append("append_axes_1", past=1000, past_max=1000, ragged=1),
        # Prompts of text and images, 12K tokens of seven sequences in all, heads-first pages, far positions.
        _append("append_axes_prompts", seqs=7, new=12000, new_max=12000, page=64, heads_first=True, cycled=True, interleaved=True,
                far=200000, ragged=2),
        # One user's drafts of five tokens: latency.  A vocabulary that fills no whole vectors.
        _verify("verify_1x5", drafts=5, drafts_max=5, vocab=100003, row=100003, ragged=3),
        # A busy server's step: 64 sequences of up to four drafts, half of them with a rejection.
        _verify("verify_64x4", seqs=64, drafts=1, drafts_max=4, rejected=0.5, ragged=4),
        # Drafts found in the text itself, so that no drafter's probabilities are there; 16-bit rows of a padded vocabulary.
        _verify("verify_256_found", seqs=256, drafts=0, drafts_max=2, vocab=50021, row=50048, dtype="bf16", drafter=False, rejected=0.7, pad=9,
                ragged=5),
        # The pages of a decode step with drafts: rejected tokens' pages are freed, the next step's taken, two users leave, two come.
        _pages("pages_step_64", "step", rows=64, length=2000, replaced=2, pages=16384, ragged=6),
        # The same for a large pool, many rows and prompts among the newcomers.
        _pages("pages_step_4096", "step", rows=4096, length=1500, replaced=300, pages=1 << 20, used=0.7, ragged=7),
        # Beams: 3 hypotheses each of 4 parents, a short cache of two layers.
        _pages("pages_fork_4x3", "fork", rows=16, parents=4, length=300, pages=1024, layers=2, used=0.4, ragged=8),
        # Many samples of each prompt, pages of 128 tokens, four layers.
        _pages("pages_fork_64x7", "fork", rows=512, parents=64, length=1500, page=128, pages=2048, layers=4, used=0.75, ragged=9),
        # The cache made dense after many users have left, so that its upper part can be given back.
        _pages("pages_compact_8k", "compact", rows=200, page=64, length=2000, pages=8192, used=0.6, layers=2, ragged=10),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "verify", "verify", "pages", "pages", "pages"])
    ragged, dtype = rng.randrange(1 << 20), rng.choice(["bf16", "bf16", "fp16"])
    axes, cycled, interleaved = rng.choice([1, 2, 3, 3, 4]), rng.random() < 0.5, rng.random() < 0.3
    base, far = rng.choice([10000.0, 500000.0]), rng.choice([0, 0, 100000, 1000000])
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 128, 192, 256])
        Hkv = rng.choice([1, 2, 4, 8, 16])
        c = _rope("drawn", n=_log(rng, 1, 32768), Hkv=Hkv, Hq=Hkv * rng.choice([1, 1, 2, 4]), d=d, rope_dim=rng.choice([d, d, d // 32 * 16]),
                  axes=axes, cycled=cycled, interleaved=interleaved, base=base, far=far, dtype=rng.choice([dtype, dtype, "fp32"]),
                  inverse=rng.random() < 0.5)
        if c["inverse"] and c["dtype"] != "fp32":
            c["out"] = rng.choice(["same", "fp32_in"])
    elif op == "append":
        d = rng.choice([64, 128, 128])
        Hkv, seqs = rng.choice([1, 2, 4, 8]), _log(rng, 1, 256)
        past_max = _log(rng, 1, 8192)
        c = _append("drawn", dtype=dtype, Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 7]), d=d, page=rng.choice([16, 32, 64, 128]),
                    heads_first=rng.random() < 0.3, seqs=seqs, past=max(0, past_max // 50 - 1), past_max=past_max,
                    new_max=_log(rng, 1, max(1, 8192 // seqs)), pad=rng.choice([0, 0, 5]), ragged=ragged, rope_dim=rng.choice([d, d, d // 2]),
                    axes=axes, cycled=cycled, interleaved=interleaved, base=base, far=far)
    elif op == "verify":
        vocab = _log(rng, 300, 200000)
        drafts_max = rng.choice([0, 1, 2, 4, 7, 16])
        c = _verify("drawn", seqs=_log(rng, 1, max(1, min(300, 40000000 // (vocab * (drafts_max + 1))))), drafts=drafts_max // 2, drafts_max=drafts_max,
                    vocab=vocab, row=vocab if rng.random() < 0.5 else -(-vocab // 64) * 64, dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    drafter=rng.random() < 0.7, rejected=rng.choice([0.0, 0.5, 1.0]), pad=rng.choice([0, 0, 3]), ragged=ragged)
    else:
        what = rng.choice(["step", "fork", "compact"])
        page = rng.choice([16, 16, 32, 64, 128])
        c = _pages("drawn", what, page=page, ragged=ragged, used=rng.choice([0.3, 0.5, 0.8]), dtype=dtype, heads_first=rng.random() < 0.3)
        if what == "step":
            c["rows"], c["length"], c["new"] = _log(rng, 1, 2048), _log(rng, 1, 4000), rng.choice([1, 2, 5, 9])
            c["replaced"] = rng.choice([0, c["rows"] // 8, c["rows"] // 2])
        elif what == "fork":
            c["parents"] = _log(rng, 1, 32)
            c["rows"], c["length"] = c["parents"] * rng.choice([2, 3, 5, 8]), _log(rng, 1, 2000)
        else:
            c["rows"], c["length"] = _log(rng, 1, 128), _log(rng, 1, 1500)
        if what != "step":
            c["layers"], c["Hkv"], c["d"] = rng.choice([1, 2, 3]), rng.choice([1, 2, 8]), rng.choice([64, 128])
        most = c["rows"] * (-(-(c["length"] + c["new"]) // page) + 1)
        c["pages"] = int(most / c["used"]) + rng.randrange(40)
    del c["name"]
    return c


def _type(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def axis_of(case):
    """The axis of each pair: by turns, or a quarter for the first axis and the rest in equal parts."""
    half, A = case["rope_dim"] // 2, case["axes"]
    if case["cycled"] or A == 1:
        return [j % A for j in range(half)]
    first = half // 4
    return [0 if j < first else min(A - 1, 1 + (j - first) * (A - 1) // (half - first)) for j in range(half)]


def frequencies(case):
    return [case["base"] ** (-2.0 * j / case["rope_dim"]) for j in range(case["rope_dim"] // 2)]


def multimodal(rng, n, axes, at):
    """Positions [axes][n] of a run of text and images that begins at `at`: all axes alike in text; in an image the first
    stands and the others run over its rows and columns."""
    parts, left = [], n
    while left > 0:
        k = min(left, rng.randint(1, 400))
        parts.append(np.tile(np.arange(at, at + k), (axes, 1)))
        at, left = at + k, left - k
        if left > 0 and axes > 1:
            h, w = rng.randint(2, 30), rng.randint(2, 30)
            k = min(left, h * w)
            i = np.arange(k)
            grid = [i // w, i % w, i % 3]
            parts.append(np.stack([np.full(k, at)] + [at + grid[a % 3] for a in range(axes - 1)]))
            at, left = at + max(h, w), left - k
    return np.concatenate(parts, 1).astype(np.int32)


def lengths(case):
    """Tokens held and new ones of each sequence of an append, drafts of each of a verification."""
    r = random.Random(case["ragged"])
    B = case["seqs"]
    if case["op"] == "verify":
        drafts = [r.randint(case["drafts"], case["drafts_max"]) for _ in range(B)]
        drafts[0] = case["drafts_max"]
        # Sequences with a rejection; one without drafts has none.
        rejected = [drafts[b] > 0 and b < math.ceil(case["rejected"] * B) for b in range(B)]
        return dict(new=[k + 1 for k in drafts], rejected=rejected, tokens=sum(drafts) + B)
    past = [r.randint(case["past"], case["past_max"]) for _ in range(B)]
    if case["new"] > 1 and case["new"] == case["new_max"]:
        cut = sorted(r.sample(range(1, case["new"]), B - 1))
        new = [b - a for a, b in zip([0] + cut, cut + [case["new"]])]
    else:
        new = [r.randint(case["new"], case["new_max"]) for _ in range(B)]
        new[0] = case["new_max"]
    return dict(past=past, new=new, kv=[a + b for a, b in zip(past, new)], tokens=sum(new))


def layout(case, seed=0):
    """The pages of a case: tables, holders, what is asked.  Lengths come from the case, which pages from the seed."""
    r = random.Random(case["ragged"])
    rng = np.random.RandomState(seed % (1 << 32))
    R, ps, P = case["rows"], case["page"], case["pages"]
    kv = [r.randint(max(1, case["length"] // 3), case["length"]) for _ in range(R)]
    if case["what"] == "fork":
        parent = [-1 if b < case["parents"] else b % case["parents"] for b in range(R)]
        tokens = [kv[p] if p >= 0 else 0 for p in parent]
        count = [-(-kv[b] // ps) if parent[b] < 0 else 0 for b in range(R)]
    else:
        parent, tokens = [-1] * R, [k + case["new"] for k in kv]
        count = [-(-k // ps) for k in (tokens if case["what"] == "step" else kv)]
        for b in r.sample(range(R), case["replaced"]):  # a user who leaves; the row's next one has as many tokens
            kv[b] = 0
    columns = max(-(-(case["length"] + case["new"]) // ps), 1) + 1
    ids = rng.permutation(P)
    table, at = np.full((R, columns), -1, np.int32), 0
    for b, k in enumerate(count):
        table[b, :k] = ids[at:at + k]
        at += k
    refs = np.zeros(P, np.int32)
    refs[ids[:at]] = 1
    # Pages that others hold, some of them several.
    others = max(0, int(case["used"] * P) - at)
    refs[ids[at:at + others]] = rng.randint(1, 4, others)
    return dict(kv=kv, parent=parent, tokens=tokens, held=count, table=table, refs=refs)


# ---------------------------------------------------------------- inputs

def _ints(v):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(v, dtype=np.int32))).cuda()


def prepare(case, seed):
    return {"rope": _prepare_rope, "append": _prepare_append, "verify": _prepare_verify, "pages": _prepare_pages}[case["op"]](case, seed)


def _normal(gen, t, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32 if math.prod(shape) < 1 << 24 else t).to(t)


def _prepare_rope(case, seed):
    gen, rng = torch.Generator(device="cuda").manual_seed(seed), random.Random(seed)
    n, Hq, Hkv, d = case["n"], case["Hq"], case["Hkv"], case["d"]
    out_t = _type(case["dtype"])
    in_t = torch.float32 if case["out"] == "fp32_in" else out_t
    s = dict(case=case, positions=_ints(multimodal(rng, n, case["axes"], case["far"])),
             freqs=torch.tensor(frequencies(case), dtype=torch.float64, device="cuda"), axis=torch.tensor(axis_of(case), device="cuda"))
    if case["inverse"]:  # the gradients are tensors of their own
        s["q"], s["k"] = _normal(gen, in_t, n, Hq, d), _normal(gen, in_t, n, Hkv, d)
    else:  # the projection writes query and key heads side by side
        qkv = _normal(gen, in_t, n, Hq + 2 * Hkv, d)
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    s["q_out"] = torch.empty(n, Hq, d, dtype=out_t, device="cuda")
    s["k_out"] = torch.empty(n, Hkv, d, dtype=out_t, device="cuda")
    if own:
        import context_long_sequence_gb300 as cpa
        s["cpa"] = cpa
        s["plan"] = cpa.RopePlan(d, case["rope_dim"], rope_axes=case["axes"], rope_axis=axis_of(case), rope_interleaved=case["interleaved"],
                                 rope_base=case["base"])
    return s


def _prepare_append(case, seed):
    gen, rng = torch.Generator(device="cuda").manual_seed(seed), random.Random(seed)
    n, ps, Hq, Hkv, d, t = lengths(case), case["page"], case["Hq"], case["Hkv"], case["d"], _type(case["dtype"])
    B, N = case["seqs"], n["tokens"] + case["pad"]
    count = [-(-k // ps) for k in n["kv"]]
    pages = sum(count) + max(2, sum(count) // 16)
    ids = np.random.RandomState(seed % (1 << 32)).permutation(pages)
    table, at = np.zeros((B, max(count)), np.int32), 0
    for b, k in enumerate(count):
        table[b, :k] = ids[at:at + k]
        at += k
    shape = (pages, Hkv, ps, d) if case["heads_first"] else (pages, ps, Hkv, d)
    k_cache, v_cache = _normal(gen, t, *shape), _normal(gen, t, *shape)
    if case["heads_first"]:
        k_cache, v_cache = k_cache.transpose(1, 2), v_cache.transpose(1, 2)
    pos = [multimodal(rng, b, case["axes"], case["far"] + a) for a, b in zip(n["past"], n["new"])]
    s = dict(case=case, k_cache=k_cache, v_cache=v_cache, q_start=_ints(np.concatenate([[0], np.cumsum(n["new"])])), kv_len=_ints(n["kv"]),
             page_table=_ints(table), tokens=n["tokens"],
             positions=_ints(np.concatenate(pos + [np.zeros((case["axes"], case["pad"]))], 1)),
             freqs=torch.tensor(frequencies(case), dtype=torch.float64, device="cuda"), axis=torch.tensor(axis_of(case), device="cuda"),
             q_out=torch.zeros(N, Hq, d, dtype=t, device="cuda"))
    qkv = _normal(gen, t, N, Hq + 2 * Hkv, d)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if own:
        import context_long_sequence_gb300 as cpa
        s["cpa"] = cpa
        s["plan"] = cpa.PagedPlan(Hq, Hkv, d, page_size=ps, dtype=t, max_seqs=B, max_tokens=N, max_new=max(n["new"]), max_pages=table.shape[1],
                                  rope_dim=case["rope_dim"], rope_base=case["base"], rope_interleaved=case["interleaved"],
                                  rope_axes=case["axes"], rope_axis=axis_of(case))
        s["cache"] = cpa.PagedCache(k_cache, v_cache)
        s["batch"] = cpa.PagedBatch(s["q_start"], s["kv_len"], s["page_table"], n_tokens=N, positions=s["positions"])
    return s


def _prepare_verify(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, V, t, B = lengths(case), case["vocab"], _type(case["dtype"]), case["seqs"]
    N = n["tokens"] + case["pad"]
    start = np.concatenate([[0], np.cumsum(n["new"])])
    # The target's probabilities, most of the vocabulary cut off as by a nucleus; the drafter's are near them, and uncut.
    logit = torch.randn(N, V, generator=gen, device="cuda") * 2.5
    p = torch.softmax(logit.masked_fill(logit < 1.0, -math.inf), -1)
    q = torch.softmax(logit + torch.randn(N, V, generator=gen, device="cuda") * 0.7, -1)
    del logit
    cut = (p == 0).float().argmax(-1)
    # Row t's draft is the token behind it.  Sequences with a rejection: drawn by the drafter, the last one a token that
    # the target has cut off.  The others: tokens that the target has too, and random numbers that accept them.
    seq = torch.from_numpy(np.repeat(np.arange(B + (case["pad"] > 0)), n["new"] + ([case["pad"]] if case["pad"] else []))).cuda()
    rejected = torch.tensor(n["rejected"] + [False], device="cuda")[seq]
    last = torch.zeros(N, dtype=torch.bool)
    last[[int(start[b + 1]) - 2 for b in range(B) if n["new"][b] > 1]] = True
    source = torch.where(rejected[:, None], q if case["drafter"] else p, p)
    drawn = torch.multinomial(source, 1, generator=gen)[:, 0]
    del source
    drawn = torch.where(rejected & last.cuda(), cut, drawn)
    u = torch.rand(N, generator=gen, device="cuda") * rejected
    tokens = torch.zeros(N, dtype=torch.int32, device="cuda")
    tokens[1:] = drawn[:-1].to(torch.int32)
    tokens[torch.from_numpy(start[:-1]).cuda()] = 1
    rows = lambda x: torch.nn.functional.pad(x, (0, case["row"] - V)).to(t)[:, :V]  # noqa: E731
    s = dict(case=case, p=rows(p), q=rows(q) if case["drafter"] else None, accept_u=u, sample_u=torch.rand(B, generator=gen, device="cuda"),
             tokens=tokens, q_start=_ints(start), kv_len=_ints([500 + k for k in n["new"]]), n_max=max(n["new"]),
             accepted=torch.zeros(B, dtype=torch.int32, device="cuda"), out=torch.full((N,), -7, dtype=torch.int32, device="cuda"),
             kv_out=torch.zeros(B, dtype=torch.int32, device="cuda"))
    if own:
        import context_long_sequence_gb300 as cpa
        s["cpa"] = cpa
        s["plan"] = cpa.PagedPlan(8, 2, 128, page_size=16, dtype=torch.bfloat16, max_seqs=B, max_tokens=N, max_new=s["n_max"], max_pages=64)
        s["batch"] = cpa.PagedBatch(s["q_start"], s["kv_len"], torch.zeros(B, 64, dtype=torch.int32, device="cuda"), n_tokens=N)
    return s


def _prepare_pages(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    a, ps, t = layout(case, seed), case["page"], _type(case["dtype"])
    R = case["rows"]
    s = dict(case=case, table=_ints(a["table"]), held=_ints(a["held"]), refs=_ints(a["refs"]), tokens=_ints(a["tokens"]),
             served=torch.zeros(R, dtype=torch.int32, device="cuda"))
    if case["what"] == "step":
        s["keep"] = _ints(a["kv"])
    elif case["what"] == "fork":
        s["parent"] = _ints(a["parent"])
        s["keep"] = _ints([-1 if p < 0 else 0 for p in a["parent"]])
    else:
        s["table_out"], s["refs_out"] = torch.full_like(s["table"], -1), torch.zeros_like(s["refs"])
        s["used"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["what"] != "step":
        inner = (case["Hkv"], ps) if case["heads_first"] else (ps, case["Hkv"])
        s["cache"] = torch.randn(case["layers"], 2, case["pages"], *inner, case["d"], generator=gen, device="cuda", dtype=t)
        if case["heads_first"]:
            s["cache"] = s["cache"].transpose(3, 4)
    if own:
        import context_long_sequence_gb300 as cpa
        s["cpa"] = cpa
        s["plan"] = cpa.PagedPlan(4 * case["Hkv"], case["Hkv"], case["d"], page_size=ps, dtype=t, max_seqs=R, max_tokens=R, max_new=1,
                                  max_pages=a["table"].shape[1])
        s["tables"] = cpa.PageTable(s["table"], s["held"])
        if case["what"] != "step":
            s["caches"] = [cpa.PagedCache(x[0], x[1]) for x in s["cache"]]
            s["moves"] = cpa.PageMoves(max(R, case["pages"] // 2))
        if case["what"] == "compact":
            s["tables_out"] = cpa.PageTable(s["table_out"], s["held"])
            s["workspace"] = cpa.alloc_pages_workspace(case["pages"])
    return s


# ---------------------------------------------------------------- plain forms

def _rotated(case, x, angle, t):
    """x [tokens][heads][d] turned by angle [tokens][pairs] (fp64), rounded to t."""
    n = case["rope_dim"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    x = x.float()
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if case["interleaved"] else (x[..., :n // 2], x[..., n // 2:n])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., n:]], -1).to(t)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"][s["axis"]].T.double() * s["freqs"]
    if c["inverse"]:
        angle = -angle
    s["q_out"].copy_(_rotated(c, s["q"], angle, s["q_out"].dtype))
    s["k_out"].copy_(_rotated(c, s["k"], angle, s["k_out"].dtype))
    return s["q_out"], s["k_out"]


def _plain_append(s):
    c = s["case"]
    t = torch.arange(s["tokens"], device="cuda")
    seq = torch.bucketize(t, s["q_start"][1:].long(), right=True)
    i = t - s["q_start"].long()[seq]
    angle = s["positions"][s["axis"]].T[t].double() * s["freqs"]
    at = s["kv_len"].long()[seq] - (s["q_start"][1:] - s["q_start"][:-1]).long()[seq] + i
    page = s["page_table"].long()[seq, at // c["page"]]
    s["q_out"][t] = _rotated(c, s["q"][t], angle, _type(c["dtype"]))
    s["k_cache"][page, at % c["page"]] = _rotated(c, s["k"][t], angle, _type(c["dtype"]))
    s["v_cache"][page, at % c["page"]] = s["v"][t]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_verify(s):
    c = s["case"]
    start, new = s["q_start"][:-1].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(s["n_max"], device="cuda")[None]
    end = s["p"].shape[0] - 1
    row = (start[:, None] + i).clamp(max=end)
    draft = s["tokens"].long()[(row + 1).clamp(max=end)]
    px = s["p"][row, draft].double()
    qx = s["q"][row, draft].double() if c["drafter"] else 1.0
    ok = (s["accept_u"][row].double() * qx < px) & (i < new[:, None] - 1)
    accepted = ok.long().cumprod(-1).sum(-1)
    rejected = accepted < new - 1
    last = start + accepted
    p = s["p"][last].double()
    if c["drafter"]:
        less = s["q"][last].double()
    else:
        less = torch.zeros_like(p).scatter_(1, s["tokens"].long()[(last + 1).clamp(max=end)][:, None], 1.0)
    w = torch.where(rejected[:, None], (p - less).clamp(min=0), p)
    sums = torch.cumsum(w, -1)
    token = (sums > s["sample_u"].double()[:, None] * sums[:, -1:]).to(torch.int8).argmax(-1)
    s["accepted"].copy_(accepted)
    s["kv_out"].copy_(s["kv_len"] - (new - 1 - accepted))
    following = torch.where(i < accepted[:, None], draft, torch.where(i == accepted[:, None], token[:, None], -1)).to(torch.int32)
    mine = i < new[:, None]
    s["out"][row[mine]] = following[mine]
    return s["accepted"], s["out"], s["kv_out"]


def _add(refs, pages, amount):
    """refs += amount at each of `pages` (-1: none), as often as it is there."""
    P = refs.shape[0]
    count = torch.zeros(P + 1, dtype=torch.int32, device=refs.device)
    pages = torch.where(pages < 0, P, pages).long().flatten()
    refs += amount * count.index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))[:P]


def _free_pages(refs):
    """Free pages in order, and how many there are."""
    P = refs.shape[0]
    free = refs == 0
    rank = torch.cumsum(free, 0) - 1
    order = torch.full((P + 1,), -1, dtype=torch.int32, device=refs.device)
    order.scatter_(0, torch.where(free, rank, P), torch.arange(P, dtype=torch.int32, device=refs.device))
    order[P] = -1
    return order, free.sum()


def _plain_resize(s, tokens):
    c, table, held, refs = s["case"], s["table"], s["held"], s["refs"]
    col = torch.arange(table.shape[1], device="cuda")[None]
    asked = tokens >= 0
    want = torch.where(asked, (tokens + c["page"] - 1) // c["page"], held)
    gone = (col >= want[:, None]) & (col < held[:, None])
    _add(refs, torch.where(gone, table, -1), -1)
    table.masked_fill_(gone, -1)
    need = (want - held).clamp(min=0)
    end = torch.cumsum(need, 0)
    order, free = _free_pages(refs)
    ok = end <= free
    k = (end - need)[:, None] + col - held[:, None]
    new = (col >= held[:, None]) & (col < want[:, None]) & ok[:, None]
    page = order[torch.where(new, k, refs.shape[0])]
    table.copy_(torch.where(new, page, table))
    _add(refs, page, 1)
    held.copy_(torch.where(ok, want, held))
    s["served"].copy_(ok)


def _plain_fork(s):
    c, table, held, refs = s["case"], s["table"], s["held"], s["refs"]
    ps = c["page"]
    col = torch.arange(table.shape[1], device="cuda")[None]
    parent, tokens = s["parent"].long(), s["tokens"]
    child = parent >= 0
    full, part = tokens // ps, tokens % ps
    need = (child & (part > 0)).int()
    end = torch.cumsum(need, 0)
    order, free = _free_pages(refs)
    ok = end <= free
    theirs = table[parent.clamp(min=0)]
    shared = (child & ok)[:, None] & (col < full[:, None])
    fresh = torch.where((need > 0) & ok, order[(end - 1).clamp(min=0)], -1)
    source = theirs.gather(1, full.clamp(max=table.shape[1] - 1)[:, None].long())[:, 0]
    _add(refs, torch.where(shared, theirs, -1), 1)
    _add(refs, fresh, 1)
    new = torch.where(shared, theirs, torch.where((fresh[:, None] >= 0) & (col == full[:, None]), fresh[:, None], table))
    table.copy_(new)
    held.copy_(torch.where(child & ok, full + need, held))
    s["served"].copy_(ok)
    rows = (fresh >= 0).nonzero()[:, 0]
    src, dst = source[rows].long(), fresh[rows].long()
    there = (torch.arange(ps, device="cuda")[None] < part[rows][:, None])[None, None, :, :, None, None]
    s["cache"][:, :, dst] = torch.where(there, s["cache"][:, :, src], s["cache"][:, :, dst])


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    P = refs.shape[0]
    page = torch.arange(P, device="cuda")
    taken = refs > 0
    used = taken.sum()
    src, dst = (taken & (page >= used)).nonzero()[:, 0], (~taken & (page < used)).nonzero()[:, 0]
    to = page.to(torch.int32)
    to[src] = dst.to(torch.int32)
    mine = torch.arange(table.shape[1], device="cuda")[None] < s["held"][:, None]
    s["table_out"].copy_(torch.where(mine, to[table.clamp(min=0).long()], s["table_out"]))
    s["refs_out"].copy_(torch.where(page < used, refs, 0))
    s["refs_out"][dst] = refs[src]
    s["used"].copy_(used)
    s["cache"][:, :, dst] = s["cache"][:, :, src]


def _plain_pages(s):
    what = s["case"]["what"]
    if what == "compact":
        _plain_compact(s)
        return s["table_out"], s["refs_out"], s["used"], s["cache"]
    _plain_resize(s, s["keep"])
    if what == "step":
        _plain_resize(s, s["tokens"])
        return s["table"], s["held"], s["refs"], s["served"]
    _plain_fork(s)
    return s["table"], s["held"], s["refs"], s["served"], s["cache"]


def _own_pages(s):
    cpa, what = s["cpa"], s["case"]["what"]
    if what == "compact":
        cpa.cp_pages_compact(s["plan"], s["refs"], [s["tables"]], s["moves"], s["workspace"], refs_out=s["refs_out"], tables_out=[s["tables_out"]],
                             used=s["used"])
        cpa.cp_pages_copy(s["plan"], s["caches"], s["caches"], s["moves"])
        return s["table_out"], s["refs_out"], s["used"], s["cache"]
    cpa.cp_pages_resize(s["plan"], s["refs"], s["tables"], s["keep"], s["served"])
    if what == "step":
        cpa.cp_pages_resize(s["plan"], s["refs"], s["tables"], s["tokens"], s["served"])
        return s["table"], s["held"], s["refs"], s["served"]
    cpa.cp_pages_fork(s["plan"], s["refs"], s["tables"], s["tables"], s["parent"], s["tokens"], s["moves"], s["served"])
    cpa.cp_pages_copy(s["plan"], s["caches"], s["caches"], s["moves"])
    return s["table"], s["held"], s["refs"], s["served"], s["cache"]


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        cpa = s["cpa"]
        if op == "rope":
            cpa.cp_rope(s["plan"], s["positions"], [s["q"], s["k"]], [s["q_out"], s["k_out"]], inverse=s["case"]["inverse"])
            return s["q_out"], s["k_out"]
        if op == "append":
            cpa.cp_cache_append(s["plan"], s["cache"], s["batch"], s["q"], s["k"], s["v"], s["q_out"])
            return s["q_out"], s["k_cache"], s["v_cache"]
        if op == "verify":
            cpa.cp_verify_drafts(s["plan"], s["batch"], s["tokens"], s["p"], s["q"], s["accept_u"], s["sample_u"], s["accepted"], s["out"],
                                 s["kv_out"])
            return s["accepted"], s["out"], s["kv_out"]
        return _own_pages(s)
    return {"rope": _plain_rope, "append": _plain_append, "verify": _plain_verify, "pages": _plain_pages}[op](s)


# ---------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "rope":
        values = case["n"] * (case["Hq"] + case["Hkv"]) * case["d"]
        size = _type(case["dtype"]).itemsize
        read = 4 if case["out"] == "fp32_in" else size
        return dict(bytes=values * (read + size) + 4 * case["n"] * case["axes"],
                    flops=3 * case["n"] * (case["Hq"] + case["Hkv"]) * case["rope_dim"])
    if op == "append":
        N, Hq, Hkv, d = lengths(case)["tokens"], case["Hq"], case["Hkv"], case["d"]
        return dict(bytes=2 * N * (Hq + 2 * Hkv) * d * 2 + 4 * N * case["axes"], flops=3 * N * (Hq + Hkv) * case["rope_dim"])
    if op == "verify":
        # One row of the target's, and one of the drafter's where a draft is rejected; a difference and a sum of each value.
        n, size = lengths(case), _type(case["dtype"]).itemsize
        rows = case["seqs"] + (sum(n["rejected"]) if case["drafter"] else 0)
        return dict(bytes=rows * case["vocab"] * size + 16 * n["tokens"] + 16 * case["seqs"], flops=2 * case["seqs"] * case["vocab"])
    a, ps = layout(case), case["page"]
    token = case["Hkv"] * case["d"] * 2 * 2 * case["layers"]  # bytes of a token's keys and values
    if case["what"] == "step":
        # What each row is asked and holds, and a table entry and a holder's count of each page freed or taken.
        pages = sum(h - -(-k // ps) for h, k in zip(a["held"], a["kv"]))
        return dict(bytes=2 * 12 * case["rows"] + 2 * 12 * pages, flops=0)
    if case["what"] == "fork":
        children = [(t // ps, t % ps) for t, p in zip(a["tokens"], a["parent"]) if p >= 0]
        # The children are dropped and forked: entries and counts of their pages, twice; the part pages read and written.
        return dict(bytes=2 * token * sum(r for _, r in children) + 2 * 16 * sum(f + 1 for f, _ in children) + 24 * case["rows"], flops=0)
    used = int((a["refs"] > 0).sum())
    moved = used * (case["pages"] - used) // case["pages"]  # of pages held here and there at random
    return dict(bytes=2 * token * ps * moved + 8 * case["pages"] + 8 * sum(a["held"]), flops=0)


# ---------------------------------------------------------------- definitions in 64 bits

def _turn(case, x, positions):
    """x [tokens][heads][d] in fp64 turned to positions [axes][tokens], as complex numbers."""
    half = case["rope_dim"] // 2
    a = np.arange(0, 2 * half, 2) if case["interleaved"] else np.arange(half)
    b = a + 1 if case["interleaved"] else a + half
    a, b = torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda()
    rate = torch.exp(-math.log(case["base"]) * torch.arange(half, dtype=torch.float64, device="cuda") / half)
    theta = torch.stack([positions[axis].double() * rate[j] for j, axis in enumerate(axis_of(case))], 1)
    if case.get("inverse"):
        theta = -theta
    w = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(theta), theta)[:, None]
    x[..., a], x[..., b] = w.real, w.imag
    return x


def exact(case, seed):
    return {"rope": _exact_rope, "append": _exact_append, "verify": _exact_verify, "pages": _exact_pages}[case["op"]](case, seed)


def _exact_rope(case, seed):
    s = _prepare_rope(case, seed)
    return _turn(case, s["q"].double(), s["positions"]), _turn(case, s["k"].double(), s["positions"])


def _exact_append(case, seed):
    s, n, ps = _prepare_append(case, seed), lengths(case), case["page"]
    q_out, kc, vc = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
    a = 0
    for b in range(case["seqs"]):
        e = a + n["new"][b]
        place = torch.arange(n["past"][b], n["kv"][b], device="cuda")
        pages = s["page_table"][b].long()[place // ps]
        q_out[a:e] = _turn(case, s["q"][a:e].double(), s["positions"][:, a:e])
        kc[pages, place % ps] = _turn(case, s["k"][a:e].double(), s["positions"][:, a:e])
        vc[pages, place % ps] = s["v"][a:e].double()
        a = e
    return q_out, kc, vc


def _exact_verify(case, seed):
    s, n = _prepare_verify(case, seed), lengths(case)
    accepted, out, kv = s["accepted"].cpu().numpy(), s["out"].cpu().numpy(), s["kv_len"].cpu().numpy()
    tokens, u, r = s["tokens"].tolist(), s["accept_u"].cpu().double().numpy(), s["sample_u"].cpu().double().numpy()
    a = 0
    for b, k in enumerate(n["new"]):
        i = 0
        while i < k - 1:
            x = tokens[a + i + 1]
            if not u[a + i] * (float(s["q"][a + i, x]) if case["drafter"] else 1.0) < float(s["p"][a + i, x]):
                break
            i += 1
        w = s["p"][a + i].double().cpu().numpy()
        if i < k - 1:
            if case["drafter"]:
                w = np.maximum(w - s["q"][a + i].double().cpu().numpy(), 0)
            else:
                w[tokens[a + i + 1]] = max(w[tokens[a + i + 1]] - 1.0, 0)
        sums = np.cumsum(w)
        accepted[b] = i
        out[a:a + k] = tokens[a + 1:a + 1 + i] + [int(np.searchsorted(sums, r[b] * sums[-1], side="right"))] + [-1] * (k - 1 - i)
        kv[b] -= k - 1 - i
        a += k
    return accepted, out, kv


def _exact_pages(case, seed):
    """The same, page by page; counts and tables as fp64 have no value of their own, so they come as they are."""
    s, a, ps = _prepare_pages(case, seed), layout(case, seed), case["page"]
    refs, table, held = a["refs"], a["table"], list(a["held"])
    P = case["pages"]
    served = np.zeros(case["rows"], np.int32)

    def moved(pairs):
        if pairs:
            src, dst, count = (torch.tensor(x, device="cuda") for x in zip(*pairs))
            for k in torch.unique(count).tolist():
                m = count == k
                s["cache"][:, :, dst[m], :k] = s["cache"][:, :, src[m], :k]

    if case["what"] == "compact":
        used = int((refs > 0).sum())
        holes = [p for p in range(used) if refs[p] == 0]
        high = [p for p in range(used, P) if refs[p] > 0]
        to = dict(zip(high, holes))
        out, refs_out = np.full_like(table, -1), refs.copy()
        for b in range(case["rows"]):
            out[b, :held[b]] = [to.get(p, p) for p in table[b, :held[b]].tolist()]
        refs_out[holes], refs_out[used:] = refs[high], 0
        moved([(x, y, ps) for x, y in to.items()])
        return out, refs_out, np.array([used], np.int32), s["cache"]

    def resize(b, want):
        while held[b] > want:
            held[b] -= 1
            refs[table[b, held[b]]] -= 1
            table[b, held[b]] = -1

    def lowest():
        at = 0
        while True:
            while at < P and refs[at] > 0:
                at += 1
            if at == P:
                return
            refs[at] = 1
            yield at

    asked = a["kv"] if case["what"] == "step" else [-1 if p < 0 else 0 for p in a["parent"]]
    for b, t in enumerate(asked):
        if t >= 0:
            resize(b, -(-t // ps))
    pages, pairs, left = lowest(), [], int((refs == 0).sum())
    for b, t in enumerate(a["tokens"]):
        p = a["parent"][b]
        if case["what"] == "step":
            resize(b, -(-t // ps))
        need = -(-t // ps) - held[b] if case["what"] == "step" else int(p >= 0 and t % ps > 0)
        need, left = max(0, need), left - max(0, need)
        served[b] = left >= 0
        if left < 0:
            continue
        if case["what"] == "fork" and p >= 0:
            full = t // ps
            table[b, :full] = table[p, :full]
            refs[table[p, :full]] += 1
            held[b] = full
            if need:
                pairs.append((int(table[p, full]), next(pages), t % ps))
                table[b, full], held[b] = pairs[-1][1], full + 1
        else:
            for _ in range(need):
                table[b, held[b]] = next(pages)
                held[b] += 1
    if case["what"] == "step":
        return table, np.array(held, np.int32), refs, served
    moved(pairs)
    return table, np.array(held, np.int32), refs, served, s["cache"]
