"""The operators between token ids and a language model, as cases that can be
timed and compared: where a batch's tokens go in a paged cache, the scores of
the next token under penalties, biases and grammar masks (with gradients), and
the token masks of a byte automaton over the vocabulary.

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
VOCABS = {"1k": "gpt2_code_1k.merges", "50k": "gpt2_mixed_50k.merges", "100k": "cl100k_session_100k.merges"}
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# --- the cases ---------------------------------------------------------------

def listed():
    return [
        # a small decode step: 64 requests append one token each to their cache
        {"name": "assign decode 64", "op": "assign", "n": 64, "max_new": 1, "max_ctx": 8000, "block": 16},
        # a large decode step, contexts of up to 32k tokens
        {"name": "assign decode 4096", "op": "assign", "n": 4096, "max_new": 1, "max_ctx": 32768, "block": 32},
        # prefill of a batch of 64 long sessions, a block size that is no power of two
        {"name": "assign prefill 64", "op": "assign", "n": 64, "max_new": 180001, "max_ctx": 3001, "block": 48},
        # a quarter of 1,000 requests ends and gives its blocks back
        {"name": "release 1000", "op": "release", "n": 1000, "max_ctx": 20011, "block": 16},
        # the prompts of 64 long sessions become the bit sets that the repetition penalty reads
        {"name": "seen bits 64", "op": "seen", "n": 64, "max_len": 180001, "n_logits": 100257},
        # one request decoding with everything on: the latency of a single token
        {"name": "logits 1 bf16", "op": "logits", "rows": 1, "n_logits": 100257, "type": "bf16", "pad": 7,
         "gen": 900, "bias": 20, "mask": True, "seen": True, "out": True},
        # an ordinary decode batch; rows of an odd number of 16-bit scores, back to back
        {"name": "logits 64 f16", "op": "logits", "rows": 64, "n_logits": 50257, "type": "f16", "pad": 0,
         "gen": 3000, "bias": 300, "mask": True, "seen": True, "out": True},
        # greedy serving: only the chosen token and its log-probability come back
        {"name": "greedy 200 f32", "op": "logits", "rows": 200, "n_logits": 100257, "type": "f32", "pad": 31,
         "gen": 500, "bias": 0, "mask": True, "seen": False, "out": False},
        # a large decode batch
        {"name": "logits 512 bf16", "op": "logits", "rows": 512, "n_logits": 100257, "type": "bf16", "pad": 63,
         "gen": 2000, "bias": 0, "mask": False, "seen": True, "out": True},
        # policy training: the gradient of 2,048 sampled tokens' log-probabilities under the same rules
        {"name": "gradient 2048 bf16", "op": "gradient", "rows": 2048, "n_logits": 50257, "type": "bf16", "pad": 47,
         "gen": 2047, "bias": 0, "mask": True, "seen": True, "dense": False},
        # one request enters a new state of its grammar
        {"name": "grammar 1", "op": "grammar", "n": 1, "vocab": "100k", "fields": 4, "every": False},
        # every state of a larger grammar at once, as when a schema is registered
        {"name": "grammar all states", "op": "grammar", "n": 0, "vocab": "100k", "fields": 20, "every": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["assign", "assign", "release", "seen", "logits", "logits", "logits", "gradient", "gradient",
                     "grammar", "grammar"])
    if op == "assign":
        n = _log(rng, 1, 4096)
        return {"op": op, "n": n, "max_new": _log(rng, 1, max(1, min(180001, 8000000 // n))),
                "max_ctx": _log(rng, 1, 32768), "block": rng.choice([1, 8, 16, 17, 32, 48, 64, 128])}
    if op == "release":
        return {"op": op, "n": _log(rng, 1, 2000), "max_ctx": _log(rng, 100, 20011), "block": rng.choice([5, 16, 32, 64])}
    if op == "seen":
        n = _log(rng, 1, 512)
        return {"op": op, "n": n, "max_len": _log(rng, 10, min(180001, 8000000 // n)),
                "n_logits": rng.choice([1257, 50257, 100257, rng.randint(300, 130000)])}
    if op in ("logits", "gradient"):
        V = rng.choice([1257, 50257, 100257, rng.randint(300, 130000)])
        kind = rng.choice(["f32", "f16", "bf16", "bf16"])
        rows = _log(rng, 1, min(2048, 400000000 // (3 * V * (4 if kind == "f32" else 2))))
        case = {"op": op, "rows": rows, "n_logits": V, "type": kind,
                "pad": rng.choice([0, 0, 7, -V % 64]), "gen": _log(rng, 1, 4000), "bias": rng.choice([0, 0, 20, 300]),
                "mask": rng.random() < 0.7, "seen": rng.random() < 0.7}
        case["out" if op == "logits" else "dense"] = rng.random() < (0.75 if op == "logits" else 0.4)
        return case
    return {"op": op, "n": _log(rng, 1, 400), "vocab": rng.choice(["1k", "50k", "100k", "100k"]),
            "fields": _log(rng, 1, 24), "every": False}


# --- inputs ------------------------------------------------------------------

@functools.lru_cache(None)
def _merges(vocab):
    with open(os.path.join(ROOT, "data", "vocabs", VOCABS[vocab]), "rb") as f:
        raw = zlib.decompress(f.read())
    n = struct.unpack_from("<4sI", raw)[1]
    return np.frombuffer(raw, "<u4", 2 * n, 8).reshape(n, 2).astype(np.uint32)


@functools.lru_cache(None)
def _tokens(vocab):
    """The token byte strings: the 256 bytes, then every merge that makes new bytes."""
    toks = [bytes([b]) for b in range(256)]
    seen = set(toks)
    for a, b in _merges(vocab).tolist():
        t = toks[a] + toks[b]
        if t not in seen:
            seen.add(t)
            toks.append(t)
    return toks


@functools.lru_cache(None)
def _tokenizer(vocab):
    """The one tokenizer that a program keeps (of the library: only where `own` is true)."""
    import exact_bpe_tokenization_utf_gb300 as pkg
    return pkg.Tokenizer(_tokens(vocab), _merges(vocab), pkg.PATTERN_CL100K)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(rng, n, most, log=True):
    """n lengths of 1..most, evenly spread (over their logarithm, or plainly), one in twenty of them 0, in an order of
    the seed's: their sum, and with it the outputs' sizes, is the same for every seed."""
    at = (np.arange(n) + 0.5) / n
    got = np.exp(at * math.log(most + 1)).astype(np.int64) if log else (at * (most + 1)).astype(np.int64)
    got = np.minimum(np.maximum(got, 1), most)
    got[19::20] = 0
    return rng.permutation(got)


def _offsets(lens):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)).cuda()


def _ids(g, n, n_logits):
    """Token ids as text has them: a few frequent ones and a long tail."""
    u = torch.rand(max(n, 1), generator=g, device="cuda")
    return (u.pow(4) * n_logits).to(torch.int32).clamp_(0, n_logits - 1)


def prepare(case, seed):
    return {"assign": _prepare_assign, "release": _prepare_release, "seen": _prepare_seen, "logits": _prepare_logits,
            "gradient": _prepare_logits, "grammar": _prepare_grammar}[case["op"]](case, seed)


def _prepare_assign(case, seed):
    rng, g = np.random.default_rng(seed), _gen(seed)
    n, block = case["n"], case["block"]
    new = _lengths(rng, n, case["max_new"])
    ctx = rng.integers(0, case["max_ctx"] + 1, n)
    total = int(new.sum())
    have, need = -(-ctx // block), -(-(ctx + new) // block)
    max_blocks = int(-(-(case["max_ctx"] + case["max_new"]) // block))
    used, spare = int(have.sum()), int((need - have).sum())
    order = torch.randperm(used + spare + 100, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n, max_blocks), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(max_blocks, device="cuda") < torch.from_numpy(have).cuda()[:, None]] = order[:used]
    cap = -(-total // 64) * 64 + 64 * (n % 2)
    s = {"case": case, "new_off": _offsets(new), "ctx": torch.from_numpy(ctx).cuda(), "table": table,
         "free": order[used:].contiguous(), "n_free": torch.tensor([spare + 100 - int(rng.integers(0, 50))], device="cuda"),
         "cap": cap}
    if own:
        import exact_bpe_tokenization_utf_gb300 as pkg
        s["slot"] = torch.empty(cap, dtype=torch.int64, device="cuda")
        s["pos"], s["req"] = (torch.empty(cap, dtype=torch.int32, device="cuda") for _ in range(2))
        s["seq_len"] = torch.empty(n, dtype=torch.int64, device="cuda")
        s["n_free_out"] = torch.empty(1, dtype=torch.int64, device="cuda")
        s["status"] = torch.empty(4, dtype=torch.int64, device="cuda")
        s["tok"] = _tokenizer("1k")
        s["args"] = pkg.PagedArgs(
            d_item_off=s["new_off"].data_ptr(), d_ctx_len=s["ctx"].data_ptr(), n=n, block_size=block,
            d_table=table.data_ptr(), table_stride=table.stride(0), max_blocks=max_blocks, d_free=s["free"].data_ptr(),
            d_n_free=s["n_free"].data_ptr(), d_n_free_out=s["n_free_out"].data_ptr(), d_slot=s["slot"].data_ptr(),
            d_pos=s["pos"].data_ptr(), d_req=s["req"].data_ptr(), cap=cap, d_seq_len=s["seq_len"].data_ptr(),
            d_status=s["status"].data_ptr())
    return s


def _prepare_release(case, seed):
    rng, g = np.random.default_rng(seed), _gen(seed)
    n, block = case["n"], case["block"]
    lens = _lengths(rng, n, case["max_ctx"], log=False)
    have = -(-lens // block)
    max_blocks = int(-(-case["max_ctx"] // block))
    used, before = int(have.sum()), 777
    order = torch.randperm(used + before, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n, max_blocks), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(max_blocks, device="cuda") < torch.from_numpy(have).cuda()[:, None]] = order[:used]
    free = torch.full((used + before + 1,), -1, dtype=torch.int32, device="cuda")
    free[:before] = order[used:]
    s = {"case": case, "lens": torch.from_numpy(lens).cuda(), "table": table, "free": free, "cap": used + before,
         "done": torch.from_numpy((rng.random(n) < 0.25).astype(np.uint8)).cuda(),
         "n_free": torch.tensor([before], device="cuda")}
    if own:
        s["n_free_out"] = torch.empty(1, dtype=torch.int64, device="cuda")
        s["status"] = torch.empty(4, dtype=torch.int64, device="cuda")
        s["tok"] = _tokenizer("1k")
    return s


def _prepare_seen(case, seed):
    rng, g = np.random.default_rng(seed), _gen(seed)
    lens = _lengths(rng, case["n"], case["max_len"])
    s = {"case": case, "off": _offsets(lens), "total": int(lens.sum()), "ids": _ids(g, int(lens.sum()), case["n_logits"])}
    if own:
        s["bits"] = torch.empty((case["n"], -(-case["n_logits"] // 32)), dtype=torch.int32, device="cuda")
        s["tok"] = _tokenizer("1k")
    return s


def _prepare_logits(case, seed):
    rng, g = np.random.default_rng(seed), _gen(seed)
    B, V = case["rows"], case["n_logits"]
    W = -(-V // 32)
    grad = case["op"] == "gradient"
    rand = lambda *size: torch.rand(*size, generator=g, device="cuda")  # noqa: E731
    store = torch.randn(B, V + case["pad"], generator=g, device="cuda").mul_(3).to(TYPES[case["type"]])
    s = {"case": case, "logits": store[:, :V], "grad": grad}
    s["repetition"], s["temperature"] = 1 + 0.5 * rand(B), 0.5 + rand(B)
    s["frequency"], s["presence"] = 0.3 * rand(B), 0.5 * rand(B)
    # what each row has generated so far: in training row b follows the first b tokens of one sequence
    if grad:
        s["gen_len"] = torch.arange(B, dtype=torch.int32, device="cuda").clamp_(max=case["gen"])
        s["gen_start"] = torch.zeros(B, dtype=torch.int64, device="cuda")
        s["gen"], s["gen_total"] = _ids(g, case["gen"], V), int(np.minimum(np.arange(B), case["gen"]).sum())
    else:
        lens = rng.integers(0, case["gen"] + 1, B)
        off = _offsets(lens)
        s["gen_len"], s["gen_start"] = torch.from_numpy(lens.astype(np.int32)).cuda(), off[:-1].clone()
        s["gen"], s["gen_total"] = _ids(g, int(lens.sum()), V), int(lens.sum())
    # the prompt's tokens, of one word in three
    words = torch.randint(-2**31, 2**31, (B, W), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    s["seen"] = torch.where(rand(B, W) < 0.33, words, 0) & words.roll(1, 1) if case["seen"] else None
    # rows inside a string allow nearly everything, rows between two fields little, some rows have no rule
    s["mask"] = None
    if case["mask"]:
        kind = rand(B, 1)
        most = torch.where(rand(B, W) < 0.9, -1, words)
        few = torch.where(rand(B, W) < 0.01, words, 0)
        few[:, W // 2] |= 1
        s["mask"] = torch.where(kind < 0.2, torch.full_like(words, -1), torch.where(kind < 0.7, most, few))
    s["bias_off"] = s["bias_id"] = s["bias"] = None
    if case["bias"]:
        k = np.minimum(_lengths(rng, B, case["bias"], log=False), V // 2)
        s["bias_off"] = _offsets(k)
        s["bias_id"] = torch.cat([torch.from_numpy(rng.choice(V, int(m), replace=False).astype(np.int32)) for m in k]
                                 + [torch.zeros(1, dtype=torch.int32)]).cuda()
        s["bias"] = 4 * torch.randn(s["bias_id"].numel(), generator=g, device="cuda")
        s["bias_n"] = int(k.sum())
    # the token whose log-probability is wanted: one that the mask allows
    u = rand(B, V) if s["mask"] is None else rand(B, V) * _unpack(s["mask"], V)
    s["pick"] = u.argmax(1).to(torch.int32)
    del u
    if grad:
        s["lse"] = _scores(s)[4]  # from the forward pass
        s["grad_logprob"] = torch.randn(B, generator=g, device="cuda")
        s["grad_out"] = None
        if case["dense"]:
            s["grad_out"] = torch.randn(B, V, generator=g, device="cuda").mul_(0.01).to(TYPES[case["type"]])
    if own:
        import exact_bpe_tokenization_utf_gb300 as pkg
        s["tok"] = _tokenizer("1k")
        p = lambda k: None if s.get(k) is None else s[k].data_ptr()  # noqa: E731
        if not grad:
            s["lse"], s["logprob"] = (torch.empty(B, device="cuda") for _ in range(2))
            s["top"] = torch.empty(B, dtype=torch.int32, device="cuda")
            s["out"] = torch.empty(B, V, dtype=TYPES[case["type"]], device="cuda") if case["out"] else None
        s["args"] = pkg.LogitsArgs(
            d_logits=s["logits"].data_ptr(), logits_stride=s["logits"].stride(0), d_out=p("out"), out_stride=V,
            dtype={"f32": pkg.DTYPE_F32, "f16": pkg.DTYPE_F16, "bf16": pkg.DTYPE_BF16}[case["type"]], rows=B, n_logits=V,
            d_seen=p("seen"), seen_stride=W, d_gen=p("gen"), d_gen_start=p("gen_start"), d_gen_len=p("gen_len"),
            d_repetition=p("repetition"), d_frequency=p("frequency"), d_presence=p("presence"),
            d_temperature=p("temperature"), d_bias_off=p("bias_off"), d_bias_id=p("bias_id"), d_bias=p("bias"),
            d_mask=p("mask"), mask_stride=W, d_pick=p("pick"), d_top=p("top"), d_lse=p("lse"), d_logprob=p("logprob"))
        if grad:
            s["grad_logits"] = torch.empty(B, V, dtype=TYPES[case["type"]], device="cuda")
            s["grad_bias"] = torch.zeros_like(s["bias"]) if case["bias"] else None
            s["grad_args"] = pkg.LogitsGradArgs(
                d_grad_out=p("grad_out"), grad_out_stride=V, d_grad_logprob=p("grad_logprob"),
                d_grad_logits=p("grad_logits"), grad_logits_stride=V, d_grad_bias=p("grad_bias"))
    return s


class _Automaton:
    """A byte automaton of JSON objects with fixed fields, built from its end to its start."""

    def __init__(self):
        self.next, self.accept, self.strings = [], [], []

    def state(self, accept=False, like=None):
        self.next.append([-1] * 256 if like is None else list(self.next[like]))
        self.accept.append(accept)
        return len(self.next) - 1

    def on(self, s, to, byts):
        for b in byts:
            self.next[s][b] = to

    def literal(self, text, to):
        for b in reversed(text):
            s = self.state()
            self.on(s, to, [b])
            to = s
        return to

    def string(self, to):
        """From inside a string to its closing quote: escapes and well-formed UTF-8."""
        st = self.state()
        c1, c2, c3, e0, ed, f0, f4, esc, h4, h3, h2, h1 = (self.state() for _ in range(12))
        tail = range(0x80, 0xC0)
        self.on(st, st, [b for b in range(32, 128) if b not in b'"\\'])
        self.on(st, to, b'"')
        for frm, dest, byts in ((st, esc, b"\\"), (esc, st, b'"\\/bfnrt'), (esc, h4, b"u"), (st, c1, range(0xC2, 0xE0)),
                                (st, c2, range(0xE1, 0xF0)), (st, e0, [0xE0]), (st, ed, [0xED]), (st, f0, [0xF0]),
                                (st, c3, range(0xF1, 0xF4)), (st, f4, [0xF4]), (c3, c2, tail), (c2, c1, tail),
                                (c1, st, tail), (e0, c1, range(0xA0, 0xC0)), (ed, c1, range(0x80, 0xA0)),
                                (f0, c2, range(0x90, 0xC0)), (f4, c2, range(0x80, 0x90))):
            self.on(frm, dest, byts)
        for frm, dest in ((h4, h3), (h3, h2), (h2, h1), (h1, st)):
            self.on(frm, dest, b"0123456789abcdefABCDEF")
        self.strings.append(st)
        return self.literal(b'"', st)

    def integer(self, to):
        digits, first, minus = self.state(like=to), self.state(), self.state()
        zero = self.state(like=to)
        self.on(digits, digits, b"0123456789")
        for s in (first, minus):
            self.on(s, digits, b"123456789")
            self.on(s, zero, b"0")
        self.on(first, minus, b"-")
        return first

    def words(self, to, words):
        s = self.state()
        for w in words:
            self.on(s, self.literal(w[1:], to), w[:1])
        return s


def _automaton(fields, rng):
    a = _Automaton()
    to = a.literal(b"}", a.state(accept=True))
    for k in range(fields):
        kind = k % 4
        to = (a.string(to) if kind in (0, 2) else a.integer(to) if kind == 1 else a.words(to, [b"true", b"false", b"null"]))
        key = bytes(rng.integers(97, 123, 3 + k * 5 % 9).astype(np.uint8))
        to = a.literal((b'{"' if k == fields - 1 else b', "') + key + b'": ', to)
    return a


def _prepare_grammar(case, seed):
    rng = np.random.default_rng(seed)
    toks = _tokens(case["vocab"])
    a = _automaton(case["fields"], rng)
    nxt, accept = np.array(a.next, dtype=np.int32), np.array(a.accept, dtype=np.uint8)
    n_states, V = len(nxt), len(toks)
    if case["every"]:
        n, states, ids = n_states, rng.permutation(n_states), np.full(n_states, -1)
    else:
        # half of the requests are inside a string, whose next token is a word; the others take one byte
        n = case["n"]
        states, ids = rng.integers(0, n_states, n), np.full(n, -1)
        plain = [t for t in range(256, V) if toks[t].isalpha() and toks[t].islower()]
        for k in range(n):
            ok = np.flatnonzero(nxt[states[k]] >= 0)
            if rng.random() < 0.5:
                states[k], ids[k] = rng.choice(a.strings), plain[int(rng.integers(0, len(plain)))]
            elif len(ok) and rng.random() < 0.9:
                ids[k] = int(rng.choice(ok))
    s = {"case": case, "n": n, "n_logits": V + 1, "eos": V, "state": torch.from_numpy(states.astype(np.int32)).cuda(),
         "ids": torch.from_numpy(ids.astype(np.int32)).cuda()}
    if own:
        import exact_bpe_tokenization_utf_gb300 as pkg
        s["grammar"] = pkg.Grammar(_tokenizer(case["vocab"]), nxt, accept)
        s["state_out"] = torch.empty_like(s["state"])
        s["mask"] = torch.empty(n, -(-(V + 1) // 32), dtype=torch.int32, device="cuda")
    else:
        # the automaton with a state for "dead" at its end, and the tokens' bytes by length
        s["next"] = torch.from_numpy(np.vstack([np.where(nxt < 0, n_states, nxt), np.full((1, 256), n_states)])).cuda()
        s["accept"] = torch.from_numpy(np.append(accept, 0)).cuda().bool()
        lens = np.array([len(t) for t in toks])
        order = np.argsort(lens, kind="stable")
        s["order"], s["lens"] = torch.from_numpy(order).cuda(), lens[order]
        byts = np.zeros((V, int(lens.max())), dtype=np.uint8)
        for k, t in enumerate(toks):
            byts[k, :len(t)] = np.frombuffer(t, np.uint8)
        s["bytes"], s["tok_len"] = torch.from_numpy(byts).cuda(), torch.from_numpy(lens).cuda()
    return s


# --- one pass ----------------------------------------------------------------

def run(state):
    return {"assign": _run_assign, "release": _run_release, "seen": _run_seen, "logits": _run_logits,
            "gradient": _run_gradient, "grammar": _run_grammar}[state["case"]["op"]](state)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _run_assign(s):
    names = ("table", "n_free_out", "slot", "pos", "req", "seq_len", "status")
    if own:
        s["tok"].paged_assign_device(s["args"], _stream())
        return {k: s[k] for k in names}
    block, off, ctx, table = s["case"]["block"], s["new_off"], s["ctx"], s["table"]
    new = off[1:] - off[:-1]
    have, need = (ctx + block - 1) // block, (ctx + new + block - 1) // block
    extra = need - have
    base = extra.cumsum(0) - extra
    t = torch.arange(s["cap"], device="cuda")
    real = t < off[-1]
    t = torch.minimum(t, off[-1] - 1)
    req = torch.searchsorted(off, t, right=True) - 1
    pos = ctx[req] + t - off[req]
    col = pos // block
    fresh = s["free"][(s["n_free"] - 1 - base[req] - (col - have[req])).clamp(0, s["free"].numel() - 1)]
    blk = torch.where(col >= have[req], fresh, table[req, col])
    table[req, col] = blk
    slot = torch.where(real, blk.to(torch.int64) * block + pos % block, -1)
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    return {"table": table, "n_free_out": s["n_free"] - extra.sum(), "slot": slot,
            "pos": torch.where(real, pos, -1).to(torch.int32), "req": torch.where(real, req, -1).to(torch.int32),
            "seq_len": ctx + new, "status": torch.cat([zero, extra.sum().reshape(1), off[-1:], zero - 1])}


def _run_release(s):
    case = s["case"]
    if own:
        t = s["table"]
        s["tok"].paged_release_device(s["lens"].data_ptr(), s["done"].data_ptr(), case["n"], case["block"], t.data_ptr(),
                                      t.stride(0), t.shape[1], s["free"].data_ptr(), s["cap"], s["n_free"].data_ptr(),
                                      s["n_free_out"].data_ptr(), s["status"].data_ptr(), _stream())
        return {"free": s["free"], "n_free_out": s["n_free_out"], "status": s["status"]}
    count = torch.where(s["done"] != 0, (s["lens"] + case["block"] - 1) // case["block"], 0)
    base = count.cumsum(0) - count
    col = torch.arange(s["table"].shape[1], device="cuda")
    to = torch.where(col < count[:, None], s["n_free"] + base[:, None] + col, s["cap"])
    s["free"].scatter_(0, to.reshape(-1), s["table"].reshape(-1))
    s["free"][-1] = -1
    n_out = s["n_free"] + count.sum()
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    return {"free": s["free"], "n_free_out": n_out, "status": torch.cat([zero, count.sum().reshape(1), zero, zero - 1])}


def _pack(bits):
    """Truth values in 32-bit words, the lowest bit first."""
    n, V = bits.shape
    W = -(-V // 32)
    full = torch.zeros(n, W * 32, dtype=torch.bool, device=bits.device)
    full[:, :V] = bits
    place = torch.arange(32, device=bits.device, dtype=torch.int64)
    return (full.view(n, W, 32).to(torch.int64) << place).sum(2).to(torch.int32)


def _unpack(words, V):
    place = torch.arange(32, device=words.device, dtype=torch.int32)
    return ((words[:, :, None] >> place) & 1).reshape(words.shape[0], -1)[:, :V].bool()


def _run_seen(s):
    case = s["case"]
    if own:
        s["tok"].seen_bits_device(s["ids"].data_ptr(), s["off"].data_ptr(), case["n"], case["n_logits"],
                                  s["bits"].data_ptr(), s["bits"].stride(0), False, _stream())
        return s["bits"]
    off = s["off"]
    row = torch.repeat_interleave(torch.arange(case["n"], device="cuda"), off[1:] - off[:-1], output_size=s["total"])
    bits = torch.zeros(case["n"], case["n_logits"], dtype=torch.bool, device="cuda")
    bits[row, s["ids"][:s["total"]].long()] = True
    return _pack(bits)


def _scores(s):
    """The rules applied in 32 bits: (factor of the repetition penalty, allowed, scores, scores over the temperature, lse)."""
    B, V = s["case"]["rows"], s["case"]["n_logits"]
    x = s["logits"].float()
    ends = s["gen_len"].to(torch.int64).cumsum(0)
    row = torch.repeat_interleave(torch.arange(B, device="cuda"), s["gen_len"], output_size=s["gen_total"])
    at = s["gen_start"][row] + torch.arange(s["gen_total"], device="cuda") - (ends - s["gen_len"])[row]
    count = torch.zeros(B, V, device="cuda")
    one = torch.ones(1, device="cuda").expand(s["gen_total"])
    count.view(-1).scatter_add_(0, row * V + s["gen"][at].long(), one)
    seen = count > 0
    if s["seen"] is not None:
        seen = seen | _unpack(s["seen"], V)
    r = s["repetition"][:, None]
    z = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    z = z - s["frequency"][:, None] * count
    z = z - s["presence"][:, None] * (count > 0)
    factor = torch.where(seen, torch.where(x > 0, 1 / r, r), 1.0)
    if s["bias_id"] is not None:
        n = s["bias_n"]
        brow = torch.repeat_interleave(torch.arange(B, device="cuda"), s["bias_off"][1:] - s["bias_off"][:-1], output_size=n)
        z[brow, s["bias_id"][:n].long()] += s["bias"][:n]
    allowed = None
    if s["mask"] is not None:
        allowed = _unpack(s["mask"], V)
        z = torch.where(allowed, z, -math.inf)
    y = z / s["temperature"][:, None]
    top = y.amax(1, keepdim=True)
    lse = (top + (y - top).exp().sum(1, keepdim=True).log())[:, 0]
    return factor, allowed, z, y, lse


def _run_logits(s):
    if own:
        s["tok"].process_logits_device(s["args"], _stream())
        got = {k: s[k] for k in ("top", "lse", "logprob")}
        if s["out"] is not None:
            got["out"] = s["out"]
        return got
    _, _, z, y, lse = _scores(s)
    top = torch.where(z.amax(1) > -math.inf, z.argmax(1), -1).to(torch.int32)
    got = {"top": top, "lse": lse, "logprob": y.gather(1, s["pick"].long()[:, None])[:, 0] - lse}
    if s["case"]["out"]:
        got["out"] = y.to(s["logits"].dtype)
    return got


def _run_gradient(s):
    if own:
        s["tok"].process_logits_backward_device(s["args"], s["grad_args"], _stream())
        got = {"grad_logits": s["grad_logits"]}
        if s["grad_bias"] is not None:
            got["grad_bias"] = s["grad_bias"]
        return got
    factor, allowed, _, y, _ = _scores(s)
    dy = (y - s["lse"][:, None]).exp() * -s["grad_logprob"][:, None]
    dy.scatter_add_(1, s["pick"].long()[:, None], s["grad_logprob"][:, None])
    if s["grad_out"] is not None:
        dy = dy + s["grad_out"].float()
    if allowed is not None:
        dy = torch.where(allowed, dy, 0.0)
    dz = dy / s["temperature"][:, None]
    got = {"grad_logits": (dz * factor).to(s["logits"].dtype)}
    if s["bias_id"] is not None:
        n = s["bias_n"]
        row = torch.repeat_interleave(torch.arange(len(dz), device="cuda"), s["bias_off"][1:] - s["bias_off"][:-1],
                                      output_size=n)
        got["grad_bias"] = torch.zeros_like(s["bias"])
        got["grad_bias"][:n] = dz[row, s["bias_id"][:n].long()]
    return got


def _run_grammar(s):
    if own:
        s["grammar"].mask_device(s["state"].data_ptr(), s["ids"].data_ptr(), None, s["n"], s["eos"],
                                 s["state_out"].data_ptr(), s["n_logits"], s["mask"].data_ptr(), s["mask"].stride(0),
                                 _stream())
        return {"state": s["state_out"], "mask": s["mask"]}
    nxt, lens, byts = s["next"].view(-1), s["lens"], s["bytes"]
    dead = s["next"].shape[0] - 1
    # each request's state after its token
    now, ids = s["state"].long(), s["ids"].long()
    length = torch.where(ids >= 0, s["tok_len"][ids.clamp(min=0)], 0)
    for p in range(byts.shape[1]):
        byte = byts[ids.clamp(min=0), p].long()
        now = torch.where(p < length, nxt[now * 256 + byte].long(), now)
    # every token walked from there, a byte at a time (a state needs the one before it): position p is left to the
    # tokens longer than p
    ordered = byts[s["order"]].long()
    at = now[:, None].expand(-1, len(lens)).to(torch.int32).contiguous()
    for p in range(byts.shape[1]):
        first = int(np.searchsorted(lens, p, side="right"))
        at[:, first:] = nxt[at[:, first:].long() * 256 + ordered[first:, p]]
    allowed = torch.zeros(len(now), s["n_logits"], dtype=torch.bool, device="cuda")
    allowed[:, s["order"]] = at != dead
    allowed[:, s["eos"]] = s["accept"][now]
    return {"state": torch.where(now == dead, -1, now).to(torch.int32), "mask": _pack(allowed)}


# --- the same in 64 bits -----------------------------------------------------

def exact(case, seed):
    if case["op"] not in ("logits", "gradient"):
        return None  # whole numbers only
    s = prepare(case, seed)
    B, V = case["rows"], case["n_logits"]
    x = s["logits"].double()
    grad = case["op"] == "gradient"
    res = torch.empty(B, V, dtype=torch.float64, device="cuda")
    lses, lps = (torch.empty(B, dtype=torch.float64, device="cuda") for _ in range(2))
    gb = None if s["bias"] is None else torch.zeros(s["bias"].numel(), dtype=torch.float64, device="cuda")
    bits = torch.arange(32, device="cuda")
    host = {k: s[k].cpu().tolist() for k in ("gen_start", "gen_len", "pick", "repetition", "frequency", "presence", "temperature")}
    off = None if gb is None else s["bias_off"].cpu().tolist()
    set_of = lambda words: (((words.long()[:, None] >> bits) & 1).reshape(-1)[:V]) == 1  # noqa: E731
    for b in range(B):
        mult = torch.ones(V, dtype=torch.float64, device="cuda")
        ids = s["gen"][host["gen_start"][b]:host["gen_start"][b] + host["gen_len"][b]].long()
        times = torch.bincount(ids, minlength=V)
        before = times > 0
        if s["seen"] is not None:
            before = before | set_of(s["seen"][b])
        r, temp = host["repetition"][b], host["temperature"][b]
        mult[before & (x[b] > 0)] = 1.0 / r
        mult[before & (x[b] <= 0)] = r
        y = x[b] * mult - host["frequency"][b] * times - host["presence"][b] * (times > 0).double()
        if off is not None:
            y.index_add_(0, s["bias_id"][off[b]:off[b + 1]].long(), s["bias"][off[b]:off[b + 1]].double())
        y = y / temp
        ok = torch.ones(V, dtype=torch.bool, device="cuda") if s["mask"] is None else set_of(s["mask"][b])
        y[~ok] = -math.inf
        lses[b] = torch.logsumexp(y, 0)
        lps[b] = y[host["pick"][b]] - lses[b]
        res[b] = y
        if grad:
            # the forward pass's own lse, as it was rounded, is an input of the gradient
            p = torch.exp(y - s["lse"][b].double())
            w = s["grad_logprob"][b].double()
            d = -w * p
            d[host["pick"][b]] += w
            if s["grad_out"] is not None:
                d += s["grad_out"][b].double()
            d = torch.where(ok, d / temp, 0.0)
            if gb is not None:
                gb[off[b]:off[b + 1]] = d[s["bias_id"][off[b]:off[b + 1]].long()]
            res[b] = d * mult
    if grad:
        return {"grad_logits": res} if gb is None else {"grad_logits": res, "grad_bias": gb}
    got = {"top": None, "lse": lses, "logprob": lps}
    if case["out"]:
        got["out"] = res
    return got


# --- what a pass cannot do without -------------------------------------------

def work(case):
    op = case["op"]
    if op == "assign":
        tokens = case["n"] * (1 if case["max_new"] == 1 else case["max_new"] / math.log(case["max_new"] + 1))
        # offsets, context lengths, sequence lengths; per token a slot, a position and a request; a table
        # entry and a free-list entry for each block
        return {"bytes": 24 * case["n"] + tokens * (16 + 8 / case["block"]), "flops": 0}
    if op == "release":
        return {"bytes": 9 * case["n"] + 8 * case["n"] * 0.25 * case["max_ctx"] / 2 / case["block"], "flops": 0}
    if op == "seen":
        return {"bytes": 4 * case["n"] * case["max_len"] / math.log(case["max_len"] + 1) + case["n"] * case["n_logits"] / 8,
                "flops": 0}
    if op in ("logits", "gradient"):
        cells, size = case["rows"] * case["n_logits"], 4 if case["type"] == "f32" else 2
        words = (case["mask"] + case["seen"]) / 8
        gen = case["gen"] * (1 if op == "gradient" else case["rows"] / 2) * 4
        moved = size * (1 + case["out"] if op == "logits" else 2 + case["dense"])
        # about six operations a score: the mask, the temperature, the maximum, the difference, its exponential, the sum
        return {"bytes": cells * (moved + words) + gen + case["rows"] * (28 + 4 * case["bias"]), "flops": 6 * cells}
    toks = _tokens(case["vocab"])
    n_states = len(_automaton(case["fields"], np.random.default_rng(0)).next)
    n = n_states if case["every"] else case["n"]
    # the vocabulary's bytes and the automaton once, a mask for each state; a step for each token's first byte
    return {"bytes": sum(map(len, toks)) + n_states * 256 * 2 + n * (len(toks) / 8 + 12), "flops": n * len(toks)}


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(k)) for k in range(6)]:
        print(c, work(c))
