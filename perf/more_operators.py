"""The operators at a language model's two ends and at its cache, as cases that
can be timed and compared: the rows of an embedding for a batch's ids and their
gradient, the keys and values of new tokens into the paged cache, the attention
of one new token over it, and the choice of the next token by temperature,
min-p, top-k and top-p.

`run` computes a case either in elementary torch operations (`own` false) or
through the library's entry points (`own` true), on the same inputs."""
import functools
import math
import os
import random
import struct
import zlib

import numpy as np
import torch

own = False

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# --- the cases ---------------------------------------------------------------

def listed():
    return [
        # a decode step of 64 requests: one token each becomes a row, scaled by the root of the width
        {"name": "embed 64", "op": "embed", "n": 64, "pad": 0, "rows": 100257, "dim": 4096, "type": "bf16",
         "out": "bf16", "scaled": True},
        # prefill of a padded batch whose token count only the device knows; 32-bit weights, 16-bit activations
        {"name": "embed 60001", "op": "embed", "n": 60001, "pad": 63, "rows": 50257, "dim": 2048, "type": "f32",
         "out": "bf16", "scaled": False},
        # the gradient of a small training batch, written whole in 32 bits
        {"name": "embed gradient 4096", "op": "embed_gradient", "n": 4096, "pad": 0, "rows": 50257, "dim": 1024,
         "type": "f32", "out": "bf16", "scaled": False},
        # the gradient of a large batch of sessions; a frequent token comes thousands of times
        {"name": "embed gradient 131057", "op": "embed_gradient", "n": 131057, "pad": 15, "rows": 100257, "dim": 2048,
         "type": "bf16", "out": "bf16", "scaled": True},
        # one request decoding: the latency of a single choice
        {"name": "sample 1 f32", "op": "sample", "rows": 1, "n_logits": 100257, "type": "f32", "pad": 0,
         "top_k": 50, "top_p": True, "min_p": False, "plain": 0.0},
        # an ordinary decode batch whose requests bring rules of their own, some of them none
        {"name": "sample 64 bf16", "op": "sample", "rows": 64, "n_logits": 50257, "type": "bf16", "pad": 7,
         "top_k": 400, "top_p": True, "min_p": True, "plain": 0.3},
        # rollouts of a large batch: top-p alone, or the whole distribution
        {"name": "sample 512 bf16", "op": "sample", "rows": 512, "n_logits": 100257, "type": "bf16", "pad": 63,
         "top_k": 0, "top_p": True, "min_p": False, "plain": 0.5},
        # a decode step's keys and values into the cache
        {"name": "store 64", "op": "store", "n": 64, "kv_heads": 8, "dim": 128, "type": "bf16", "block": 16,
         "layout": "token", "pad": 0},
        # a prefill's, padded, into a cache that keeps a head's tokens of a block together
        {"name": "store 16381", "op": "store", "n": 16381, "kv_heads": 8, "dim": 128, "type": "f16", "block": 32,
         "layout": "head", "pad": 3},
        # one request with a long context: the latency of its attention
        {"name": "attend 1", "op": "attend", "n": 1, "most": 32749, "even": True, "kv_heads": 8, "group": 4, "dim": 128,
         "type": "bf16", "block": 16, "layout": "token", "window": 0},
        # an ordinary decode batch: short and long contexts, one key head for several queries' heads
        {"name": "attend 64", "op": "attend", "n": 64, "most": 16381, "even": False, "kv_heads": 8, "group": 5,
         "dim": 128, "type": "f16", "block": 48, "layout": "head", "window": 0},
        # a large decode batch
        {"name": "attend 256", "op": "attend", "n": 256, "most": 4801, "even": True, "kv_heads": 8, "group": 8,
         "dim": 128, "type": "bf16", "block": 16, "layout": "token", "window": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_gradient", "embed_gradient", "sample", "sample", "sample", "store", "attend",
                     "attend", "attend"])
    kind = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op in ("embed", "embed_gradient"):
        rows = rng.choice([1257, 50257, 100257, rng.randint(300, 130000)])
        dim = rng.choice([768, 1024, 2048, 4096, rng.randint(1, 1200), 8 * rng.randint(1, 300)])
        # the whole gradient, or the rows, stay below the listed ones' bytes
        dim = min(dim, max(1, 500000000 // (rows * SIZE[kind])))
        n = _log(rng, 1, min(131072, 480000000 // (dim * 4)))
        return {"op": op, "n": n, "pad": rng.choice([0, 0, 1, 63]), "rows": rows, "dim": dim, "type": kind,
                "out": rng.choice([kind, "bf16", "f16", "f32"]), "scaled": rng.random() < 0.5}
    if op == "sample":
        V = rng.choice([1257, 50257, 100257, rng.randint(300, 130000)])
        rows = _log(rng, 1, min(512, 100000000 // (V * SIZE[kind])))
        return {"op": op, "rows": rows, "n_logits": V, "type": kind, "pad": rng.choice([0, 0, 7, -V % 64]),
                "top_k": rng.choice([0, 1, 50, 400, V // 3]), "top_p": rng.random() < 0.6, "min_p": rng.random() < 0.4,
                "plain": rng.choice([0.0, 0.3, 1.0])}
    kind = rng.choice(["f16", "bf16", "bf16"])
    case = {"op": op, "n": 1, "kv_heads": rng.choice([1, 2, 4, 8, 8]), "dim": rng.choice([64, 80, 96, 128, 128, 256]),
            "type": kind, "block": rng.choice([1, 8, 16, 16, 32, 48, 64, 128]), "layout": rng.choice(["token", "head"])}
    token = 2 * 2 * case["kv_heads"] * case["dim"]
    if op == "store":
        case.update(n=_log(rng, 1, min(16384, 67000000 // token)), pad=rng.choice([0, 0, 1, 63]))
        return case
    n = _log(rng, 1, 256)
    most = _log(rng, 1, min(32768, 2400000000 // (n * token)))
    case.update(n=n, most=most, even=rng.random() < 0.4, group=rng.choice([1, 2, 4, 5, 7, 8, 8, 12, 16]),
                window=rng.choice([0, 0, 0, 1, 1024, rng.randint(1, 8192)]))
    return case


# --- inputs ------------------------------------------------------------------

@functools.lru_cache(None)
def _tokenizer():
    """The one tokenizer that a program keeps (of the library: only where `own` is true)."""
    import exact_bpe_tokenization_utf_gb300 as pkg
    with open(os.path.join(ROOT, "data", "vocabs", "gpt2_code_1k.merges"), "rb") as f:
        raw = zlib.decompress(f.read())
    n = struct.unpack_from("<4sI", raw)[1]
    return pkg.Tokenizer.from_merges(np.frombuffer(raw, "<u4", 2 * n, 8).reshape(n, 2).astype(np.uint32), pkg.PATTERN_GPT2)


def _code(kind):
    import exact_bpe_tokenization_utf_gb300 as pkg
    return {"f32": pkg.DTYPE_F32, "f16": pkg.DTYPE_F16, "bf16": pkg.DTYPE_BF16}[kind]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, kind, *size):
    return torch.randn(*size, generator=g, device="cuda", dtype=TYPES[kind])


def _ids(g, n, n_rows):
    """Token ids as text has them: a few frequent ones and a long tail."""
    u = torch.rand(max(n, 1), generator=g, device="cuda", dtype=torch.float64)
    return (u.pow(4) * n_rows).to(torch.int32).clamp_(0, n_rows - 1)


def _scale(case):
    return float(np.float32(math.sqrt(case["dim"]))) if case["scaled"] else 1.0


def _lengths(case):
    """The requests' lengths, 0 to `most`: evenly spread, or over their logarithm; the same for every seed."""
    at = (np.arange(case["n"]) + 0.5) / case["n"]
    most = case["most"]
    if case["n"] == 1:
        return np.array([most])
    got = (at * (most + 1)).astype(np.int64) if case["even"] else np.exp(at * math.log(most + 1)).astype(np.int64)
    return np.minimum(got, most)


def prepare(case, seed):
    return {"embed": _prepare_embed, "embed_gradient": _prepare_embed, "sample": _prepare_sample,
            "store": _prepare_store, "attend": _prepare_attend}[case["op"]](case, seed)


def _prepare_embed(case, seed):
    g = _gen(seed)
    n, cap, V, dim = case["n"], case["n"] + case["pad"], case["rows"], case["dim"]
    grad = case["op"] == "embed_gradient"
    s = {"case": case, "ids": _ids(g, cap, V), "n": torch.tensor([n], dtype=torch.int64, device="cuda")}
    # one token in 200 has no row: an image's place, or padding inside the batch
    s["ids"][torch.rand(cap, generator=g, device="cuda") < 0.005] = -1
    if grad:
        s["grad_out"] = _randn(g, case["out"], cap, dim).mul_(0.01)
    else:
        s["weight"] = _randn(g, case["type"], V, dim).mul_(0.02)
    if own:
        import exact_bpe_tokenization_utf_gb300 as pkg
        tok = s["tok"] = _tokenizer()
        count = s["n"].data_ptr() if case["pad"] else None
        if grad:
            s["grad_weight"] = torch.zeros(V, dim, dtype=TYPES[case["type"]], device="cuda")
            size = tok.embed_work_bytes(cap, V, dim)
            s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda")
            s["args"] = pkg.EmbedGradArgs(
                d_ids=s["ids"].data_ptr(), n=cap, d_n=count, n_rows=V, dim=dim, scale=_scale(case),
                d_grad_out=s["grad_out"].data_ptr(), grad_out_stride=dim, grad_out_dtype=_code(case["out"]),
                d_grad_weight=s["grad_weight"].data_ptr(), grad_weight_stride=dim, grad_weight_dtype=_code(case["type"]),
                accumulate=0, d_work=s["work"].data_ptr(), work_bytes=size)
        else:
            s["out"] = torch.zeros(cap, dim, dtype=TYPES[case["out"]], device="cuda")
            s["args"] = pkg.EmbedArgs(
                d_ids=s["ids"].data_ptr(), n=cap, d_n=count, n_rows=V, dim=dim, scale=_scale(case),
                d_weight=s["weight"].data_ptr(), weight_stride=dim, weight_dtype=_code(case["type"]),
                d_out=s["out"].data_ptr(), out_stride=dim, out_dtype=_code(case["out"]))
    return s


def _prepare_sample(case, seed):
    g = _gen(seed)
    B, V = case["rows"], case["n_logits"]
    rand = lambda *size: torch.rand(*size, generator=g, device="cuda")  # noqa: E731
    # a model's scores: a broad bulk and a few tokens far above it, some rows surer than others
    x = torch.randn(B, V + case["pad"], generator=g, device="cuda").mul_(2.2)
    lift = -torch.log(1 - rand(B, 64)) * (1 + 4 * rand(B, 1))
    x.scatter_add_(1, torch.randint(0, V, (B, 64), generator=g, device="cuda"), lift)
    # one row in five is under a grammar that allows little
    few = (rand(B, 1) < 0.2) & (rand(B, V + case["pad"]) > 0.02)
    few[:, V // 2] = False
    s = {"case": case, "scores": x.masked_fill_(few, -math.inf).to(TYPES[case["type"]])[:, :V]}
    del x, few
    # requests without rules keep the whole distribution
    free = rand(B) < case["plain"]
    s["temperature"] = 0.4 + rand(B)
    s["random"] = rand(B)
    s["top_k"] = s["top_p"] = s["min_p"] = None
    if case["top_k"]:
        k = (case["top_k"] * (0.2 + 0.8 * rand(B))).ceil().to(torch.int32)
        s["top_k"] = torch.where(free, 0, k)
    if case["top_p"]:
        s["top_p"] = torch.where(free, 1.0, 0.8 + 0.19 * rand(B))
    if case["min_p"]:
        s["min_p"] = torch.where(free | (rand(B) < 0.5), 0.0, 0.01 + 0.1 * rand(B))
    if own:
        import exact_bpe_tokenization_utf_gb300 as pkg
        s["tok"] = _tokenizer()
        s["pick"], s["kept"] = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
        s["logprob"] = torch.empty(B, device="cuda")
        p = lambda k: None if s[k] is None else s[k].data_ptr()  # noqa: E731
        s["args"] = pkg.SampleArgs(
            d_scores=s["scores"].data_ptr(), scores_stride=s["scores"].stride(0), dtype=_code(case["type"]), rows=B,
            n_logits=V, d_temperature=p("temperature"), d_min_p=p("min_p"), d_top_k=p("top_k"), d_top_p=p("top_p"),
            d_random=p("random"), d_pick=p("pick"), d_kept=p("kept"), d_logprob=p("logprob"))
    return s


def _cache(g, case, n_blocks):
    """Keys and values as [block, place, head, width], with one block more than the cache has, and its strides."""
    H, bs, D = case["kv_heads"], case["block"], case["dim"]
    size = (n_blocks + 1, bs, H, D) if case["layout"] == "token" else (n_blocks + 1, H, bs, D)
    both = [_randn(g, case["type"], *size) for _ in range(2)]
    return both if case["layout"] == "token" else [t.transpose(1, 2) for t in both]


def _cache_struct(s):
    import exact_bpe_tokenization_utf_gb300 as pkg
    k, case = s["k"], s["case"]
    return pkg.KVCache(d_k=k.data_ptr(), d_v=s["v"].data_ptr(), block_stride=k.stride(0), token_stride=k.stride(1),
                       head_stride=k.stride(2), dtype=_code(case["type"]), n_blocks=k.shape[0] - 1,
                       block_size=case["block"], kv_heads=case["kv_heads"], head_dim=case["dim"])


def _prepare_store(case, seed):
    g = _gen(seed)
    n, H, bs, D = case["n"], case["kv_heads"], case["block"], case["dim"]
    n_blocks = -(-n // bs) * 5 // 4 + 1
    s = {"case": case}
    s["k"], s["v"] = _cache(g, case, n_blocks)
    # queries, keys and values as one product writes them: a token's keys, then its values
    s["new"] = _randn(g, case["type"], n + case["pad"], 2 * H, D)
    if bs == 1 or n <= 256:   # a decode step: anywhere
        slot = torch.randperm(n_blocks * bs, generator=g, device="cuda")[:n]
    else:                     # a prefill: whole blocks
        blocks = torch.randperm(n_blocks, generator=g, device="cuda")
        at = torch.arange(n, device="cuda")
        slot = blocks[at // bs] * bs + at % bs
    s["slot"] = torch.cat([slot, torch.full((case["pad"],), -1, device="cuda")])
    if own:
        import exact_bpe_tokenization_utf_gb300 as pkg
        s["tok"], s["cache"] = _tokenizer(), _cache_struct(s)
        new = s["new"]
        s["args"] = pkg.StoreArgs(d_k=new.data_ptr(), d_v=new[:, H:].data_ptr(), token_stride=new.stride(0),
                                  head_stride=new.stride(1), d_slot=s["slot"].data_ptr(), n=n + case["pad"])
    return s


def _prepare_attend(case, seed):
    rng, g = np.random.default_rng(seed), _gen(seed)
    n, H, bs, D = case["n"], case["kv_heads"], case["block"], case["dim"]
    heads = H * case["group"]
    lens = rng.permutation(_lengths(case))
    have = -(-lens // bs)
    n_blocks, max_blocks = int(have.sum()) + 3, int(have.max()) + 1
    s = {"case": case, "lens": lens.tolist()}
    s["k"], s["v"] = _cache(g, case, n_blocks)
    s["q"] = _randn(g, case["type"], n, heads, D).mul_(1 + 2 * torch.rand(n, heads, 1, generator=g, device="cuda"))
    order = torch.randperm(n_blocks, generator=g, device="cuda").to(torch.int32)
    s["table"] = torch.full((n, max_blocks), -1, dtype=torch.int32, device="cuda")
    there = torch.arange(max_blocks, device="cuda") < torch.from_numpy(have).cuda()[:, None]
    s["table"][there] = order[:int(have.sum())]
    s["seq_len"] = torch.from_numpy(lens).cuda()
    if own:
        import exact_bpe_tokenization_utf_gb300 as pkg
        tok = s["tok"] = _tokenizer()
        s["cache"] = _cache_struct(s)
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(n, heads, device="cuda")
        size = tok.attend_work_bytes(n, heads, H, D)
        s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        s["args"] = pkg.AttendArgs(
            d_q=s["q"].data_ptr(), q_stride=s["q"].stride(0), q_head_stride=D, d_out=s["out"].data_ptr(),
            out_stride=s["out"].stride(0), out_head_stride=D, d_lse=s["lse"].data_ptr(), n=n, heads=heads,
            scale=float(np.float32(D ** -0.5)), window=case["window"], d_table=s["table"].data_ptr(),
            table_stride=max_blocks, max_blocks=max_blocks, d_seq_len=s["seq_len"].data_ptr(),
            d_work=s["work"].data_ptr(), work_bytes=size)
    return s


# --- one pass ----------------------------------------------------------------

def run(state):
    return {"embed": _run_embed, "embed_gradient": _run_embed_gradient, "sample": _run_sample, "store": _run_store,
            "attend": _run_attend}[state["case"]["op"]](state)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _run_embed(s):
    if own:
        s["tok"].embed_device(s["args"], _stream())
        return s["out"]
    case, ids = s["case"], s["ids"]
    there = (ids >= 0) & (torch.arange(len(ids), device="cuda") < s["n"])
    rows = s["weight"][ids.clamp(min=0).long()].float() * _scale(case)
    return torch.where(there[:, None], rows, 0.0).to(TYPES[case["out"]])


def _run_embed_gradient(s):
    if own:
        s["tok"].embed_backward_device(s["args"], _stream())
        return s["grad_weight"]
    case, ids = s["case"], s["ids"]
    there = (ids >= 0) & (torch.arange(len(ids), device="cuda") < s["n"])
    # a frequent token's sum is long: 64 bits
    total = torch.zeros(case["rows"] + 1, case["dim"], dtype=torch.float64, device="cuda")
    total.index_add_(0, torch.where(there, ids, case["rows"]).long(), s["grad_out"].double())
    return (total[:-1] * _scale(case)).to(TYPES[case["type"]])


def _run_sample(s):
    if own:
        s["tok"].sample_device(s["args"], _stream())
        return {k: s[k] for k in ("pick", "kept", "logprob")}
    # which tokens are kept and which one is chosen are decided next to borders: 64 bits
    x, order = s["scores"].double().sort(dim=1, descending=True, stable=True)   # (equal scores by their ids)
    w = ((x - x[:, :1]) / s["temperature"].double()[:, None]).exp()
    keep = x > -math.inf
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    if s["top_k"] is not None:
        k = torch.where(s["top_k"] > 0, s["top_k"], x.shape[1])
        keep &= torch.arange(x.shape[1], device="cuda") < k[:, None]
    del x
    w = torch.where(keep, w, 0.0)
    upto = w.cumsum(1)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        before = torch.cat([torch.zeros_like(upto[:, :1]), upto[:, :-1]], 1)
        keep &= (before < p * upto[:, -1:]) | (p >= 1)
        del before
    kept = keep.sum(1)
    total = upto.gather(1, (kept - 1).clamp(min=0)[:, None])
    at = (upto <= s["random"].double()[:, None] * total).sum(1).clamp(max=kept - 1)[:, None]
    logprob = (w.gather(1, at) / total).log()
    return {"pick": order.gather(1, at)[:, 0].to(torch.int32), "kept": kept.to(torch.int32),
            "logprob": logprob[:, 0].float()}


def _run_store(s):
    k, v = s["k"], s["v"]
    if own:
        s["tok"].paged_store_device(s["cache"], s["args"], _stream())
        return {"k": k[:-1], "v": v[:-1]}
    H, bs = s["case"]["kv_heads"], s["case"]["block"]
    slot = torch.where(s["slot"] < 0, (k.shape[0] - 1) * bs, s["slot"])   # (the block that the cache does not have)
    k[slot // bs, slot % bs] = s["new"][:, :H]
    v[slot // bs, slot % bs] = s["new"][:, H:]
    return {"k": k[:-1], "v": v[:-1]}


def _run_attend(s):
    if own:
        s["tok"].paged_attend_device(s["cache"], s["args"], _stream())
        return {"out": s["out"], "lse": s["lse"]}
    case, q = s["case"], s["q"]
    H, bs, D = case["kv_heads"], case["block"], case["dim"]
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, device="cuda")
    for r, m in enumerate(s["lens"]):
        if m == 0:
            continue
        at = torch.arange(max(0, m - case["window"]) if case["window"] else 0, m, device="cuda")
        block = s["table"][r, at // bs].long()
        k, v = (t[block, at % bs].float() for t in (s["k"], s["v"]))                       # [tokens, key heads, width]
        x = torch.einsum("hgd,thd->hgt", q[r].view(H, -1, D).float(), k) * D ** -0.5
        top = x.amax(2, keepdim=True)
        w = (x - top).exp()
        total = w.sum(2, keepdim=True)
        out[r] = (torch.einsum("hgt,thd->hgd", w, v) / total).reshape(-1, D).to(q.dtype)
        lse[r] = (top + total.log()).reshape(-1)
    return {"out": out, "lse": lse}


# --- the same in 64 bits -----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "embed_gradient": _exact_embed_gradient, "sample": _exact_sample,
            "store": lambda s: None, "attend": _exact_attend}[case["op"]](s)   # (a copy computes nothing)


def _exact_embed(s):
    case = s["case"]
    out = torch.zeros(len(s["ids"]), case["dim"], dtype=torch.float64, device="cuda")
    rows = torch.nonzero(s["ids"][:case["n"]] >= 0)[:, 0]
    for part in rows.split(8192):
        out[part] = s["weight"].index_select(0, s["ids"][part]).double() * _scale(case)
    return out


def _exact_embed_gradient(s):
    case = s["case"]
    ids = s["ids"][:case["n"]].long()
    place = torch.argsort(ids, stable=True)
    place = place[int((ids < 0).sum()):]
    total = torch.zeros(case["rows"], case["dim"], dtype=torch.float64, device="cuda")
    if not len(place):
        return total
    have, count = torch.unique_consecutive(ids[place], return_counts=True)
    ends = count.cumsum(0)
    # sums over runs of equal ids, a few columns at a time
    for c in range(0, case["dim"], 256):
        part = s["grad_out"][:, c:c + 256].double()[place]
        run = torch.repeat_interleave(torch.arange(len(have), device="cuda"), count, output_size=int(ends[-1]))
        at = torch.zeros(len(have), part.shape[1], dtype=torch.float64, device="cuda").index_add(0, run, part)
        total[have, c:c + 256] = at * _scale(case)
    return total


def _exact_sample(s):
    x = s["scores"].double()
    B = x.shape[0]
    host = {k: None if s[k] is None else s[k].cpu().tolist() for k in ("temperature", "random", "top_k", "top_p", "min_p")}
    lp = torch.empty(B, dtype=torch.float64, device="cuda")
    for b in range(B):
        y = x[b] / host["temperature"][b]
        ids = torch.nonzero(y > -math.inf)[:, 0]
        ids = ids[torch.argsort(-y[ids], stable=True)]
        prob = torch.softmax(y[ids], 0)
        if host["min_p"] is not None:
            ids = ids[prob >= host["min_p"][b] * prob[0]]
        if host["top_k"] is not None and host["top_k"][b] > 0:
            ids = ids[:host["top_k"][b]]
        prob = torch.softmax(y[ids], 0)
        if host["top_p"] is not None and host["top_p"][b] < 1:
            n = int(torch.searchsorted(prob.cumsum(0), torch.tensor([host["top_p"][b]], dtype=torch.float64, device="cuda")))
            ids = ids[:n + 1]
            prob = torch.softmax(y[ids], 0)
        at = int(torch.searchsorted(prob.cumsum(0), torch.tensor([host["random"][b]], dtype=torch.float64, device="cuda"),
                                    right=True))
        lp[b] = prob[min(at, len(ids) - 1)].log()
    return {"pick": None, "kept": None, "logprob": lp}


def _exact_attend(s):
    case = s["case"]
    G, bs, D = case["group"], case["block"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for r, m in enumerate(s["lens"]):
        first = max(0, m - case["window"]) if case["window"] else 0
        if m == 0:
            continue
        blocks = s["table"][r, first // bs:-(-m // bs)].long()
        cut = slice(first - first // bs * bs, m - first // bs * bs)
        for h in range(case["kv_heads"]):
            k, v = (t[blocks, :, h].reshape(-1, D)[cut].double() for t in (s["k"], s["v"]))
            y = s["q"][r, h * G:(h + 1) * G].double() @ k.t() / math.sqrt(D)
            lse[r, h * G:(h + 1) * G] = torch.logsumexp(y, 1)
            out[r, h * G:(h + 1) * G] = torch.softmax(y, 1) @ v
    return {"out": out, "lse": lse}


# --- what a pass cannot do without -------------------------------------------

def _distinct(n, rows):
    """How many of the rows n ids of _ids name, on average."""
    edge = (np.arange(rows + 1) / rows) ** 0.25
    return float((1 - (1 - np.diff(edge)) ** n).sum())


def work(case):
    op = case["op"]
    if op in ("embed", "embed_gradient"):
        n, V, dim = case["n"], case["rows"], case["dim"]
        if op == "embed":   # ids, each row that is named, what is written
            return {"bytes": 4 * n + dim * (SIZE[case["type"]] * _distinct(n, V) + SIZE[case["out"]] * n), "flops": n * dim}
        return {"bytes": 4 * n + dim * (SIZE[case["out"]] * n + SIZE[case["type"]] * V), "flops": n * dim}
    if op == "sample":
        # a score's difference, exponential and sum, and two comparisons
        cells = case["rows"] * case["n_logits"]
        return {"bytes": cells * SIZE[case["type"]] + 32 * case["rows"], "flops": 6 * cells}
    token = 2 * 2 * case["kv_heads"] * case["dim"]   # a token's keys and values
    if op == "store":
        return {"bytes": case["n"] * (2 * token + 8), "flops": 0}
    lens = _lengths(case)
    tokens = int(np.minimum(lens, case["window"]).sum() if case["window"] else lens.sum())
    heads = case["kv_heads"] * case["group"]
    return {"bytes": tokens * (token + 4 / case["block"]) + case["n"] * heads * (4 * case["dim"] + 4),
            "flops": 4 * tokens * heads * case["dim"]}


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(k)) for k in range(6)]:
        print(c, work(c))
