"""tok_paged_assign and tok_paged_release against plain loops: every output is
a whole number and has to be equal.  Lengths of 0 and 1, many requests inside
a tile of tokens and many tiles inside a request, block sizes of 1 and odd
ones, padding, in-place counters, and the errors that only the device sees."""
import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    from exact_bpe_tokenization_utf_gb300 import _build
    _build.build()
    import exact_bpe_tokenization_utf_gb300 as pkg
    tok = pkg.Tokenizer.from_merges([], pkg.PATTERN_GPT2)
    yield torch, pkg, tok
    tok.close()


def _blocks(n, bs):
    return -(-n // bs)


def _expected(new, ctx, bs, table, free, n_free, cap):
    """The definition, request by request; (table, slot, pos, req, seq_len, n_free)."""
    table, slot, pos, req = table.copy(), [], [], []
    for k, (m, c) in enumerate(zip(new, ctx)):
        have, need = _blocks(c, bs), _blocks(c + m, bs)
        for j in range(have, need):
            n_free -= 1
            table[k, j] = free[n_free]
        p = np.arange(c, c + m)
        slot.append(table[k, p // bs].astype(np.int64) * bs + p % bs if m else np.zeros(0, np.int64))
        pos.append(p)
        req.append(np.full(m, k))
    pad = np.full(cap - int(sum(new)), -1)
    cat = lambda parts: np.concatenate(parts + [pad])  # noqa: E731
    return table, cat(slot), cat(pos), cat(req), np.asarray(ctx) + np.asarray(new), n_free


class _Call:
    def __init__(self, torch, pkg, new, ctx, bs, max_blocks=None, spare=3, pad=5, n_free=None, stride_pad=0, seed=0, cap=None):
        rng = np.random.default_rng(seed)
        self.torch, self.pkg, self.new, self.bs = torch, pkg, list(new), bs
        self.ctx = [0] * len(new) if ctx is None else list(ctx)
        have = [_blocks(c, bs) for c in self.ctx]
        need = [_blocks(c + m, bs) for c, m in zip(self.ctx, new)]
        self.max_blocks = max(need + [1]) if max_blocks is None else max_blocks
        order = rng.permutation(sum(need) + spare).astype(np.int32)
        self.table = np.full((len(new), self.max_blocks + stride_pad), -1, dtype=np.int32)
        at = 0
        for k, m in enumerate(have):
            self.table[k, :m] = order[at:at + m][:self.max_blocks]
            at += m
        self.free = order[at:].copy()
        self.n_free = len(self.free) if n_free is None else n_free
        self.taken = sum(need) - sum(have)
        self.total = sum(new)
        self.cap = self.total + pad if cap is None else cap
        dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a).astype(t)).cuda()  # noqa: E731
        self.d = {"off": dev(np.concatenate([[0], np.cumsum(new)]), np.int64),
                  "ctx": None if ctx is None else dev(self.ctx, np.int64), "table": dev(self.table, np.int32),
                  "free": dev(self.free if len(self.free) else [0], np.int32), "n_free": dev([self.n_free], np.int64),
                  "n_free_out": dev([-7], np.int64), "seq": dev([-7] * len(new), np.int64),
                  "status": dev([-7] * 4, np.int64)}
        # two guard entries behind each array
        for name, t in (("slot", torch.int64), ("pos", torch.int32), ("req", torch.int32)):
            self.d[name] = torch.full((self.cap + 2,), -9, dtype=t, device="cuda")

    def args(self, **other):
        p = lambda k: None if self.d[k] is None else self.d[k].data_ptr()  # noqa: E731
        f = dict(d_item_off=p("off"), d_ctx_len=p("ctx"), n=len(self.new), block_size=self.bs, d_table=p("table"),
                 table_stride=self.table.shape[1], max_blocks=self.max_blocks, d_free=p("free"), d_n_free=p("n_free"),
                 d_n_free_out=p("n_free_out"), d_slot=p("slot"), d_pos=p("pos"), d_req=p("req"), cap=self.cap,
                 d_seq_len=p("seq"), d_status=p("status"))
        f.update(other)
        return self.pkg.PagedArgs(**f)

    def host(self, k):
        return self.d[k].cpu().numpy()

    def check(self, n_free="n_free_out", seq="seq"):
        table, slot, pos, req, lens, left = _expected(self.new, self.ctx, self.bs, self.table, self.free, self.n_free, self.cap)
        assert self.host("status").tolist() == [0, self.taken, self.total, -1]
        assert np.array_equal(self.host("table"), table)
        for name, want in (("slot", slot), ("pos", pos), ("req", req)):
            got = self.host(name)
            assert np.array_equal(got[:self.cap], want), name
            assert (got[self.cap:] == -9).all()
        assert self.host(n_free).tolist() == [left]
        assert np.array_equal(self.host(seq), lens)

    def check_refused(self, code, bad):
        st = self.host("status").tolist()
        assert st[0] == code and st[3] == bad
        assert np.array_equal(self.host("table"), self.table)
        for name in ("slot", "pos", "req"):
            got = self.host(name)
            assert (got[:self.cap] == -1).all() and (got[self.cap:] == -9).all()
        assert self.host("n_free_out").tolist() == [self.n_free]
        assert np.array_equal(self.host("seq"), self.ctx)
        return st


def _mixed(seed, n, most_new, most_ctx):
    rng = np.random.default_rng(seed)
    new = rng.integers(0, most_new + 1, n)
    new[rng.random(n) < 0.3] = 0
    return new.tolist(), rng.integers(0, most_ctx + 1, n).tolist()


SHAPES = [
    ("one token", [1], [0], 1), ("no token", [0], [5], 4), ("block edges", [1, 1, 1, 1], [15, 16, 17, 0], 16),
    ("fills a block", [16, 15, 17], [0, 1, 15], 16), ("no contexts", [3, 0, 40], None, 7),
    ("empty requests around", [0, 0, 5, 0, 0, 7, 0], [3, 0, 0, 9, 1, 2, 0], 3),
    ("tile edges", [1023, 1, 1024, 1025, 2048, 1], [0, 7, 1, 0, 3, 0], 64),
    ("one long", [500_000], [12_345], 48), ("block of one", [700, 3], [0, 300], 1),
    ("large block", [3000, 10], [1, 1 << 19], 1 << 20),
] + [("mixed %d" % s, *_mixed(s, *m), bs) for s, m, bs in (
    (1, (3000, 1, 500), 16), (2, (700, 30, 100), 5), (3, (64, 20_000, 3000), 48), (4, (9000, 3, 64), 32))]


@pytest.mark.parametrize("new,ctx,bs", [s[1:] for s in SHAPES], ids=[s[0] for s in SHAPES])
def test_assign(env, new, ctx, bs):
    torch, pkg, tok = env
    c = _Call(torch, pkg, new, ctx, bs, stride_pad=3, seed=len(new))
    tok.paged_assign_device(c.args(), torch.cuda.current_stream().cuda_stream)
    c.check()
    # again with the exact number of free blocks, in place, without the optional outputs
    c = _Call(torch, pkg, new, ctx, bs, spare=0, pad=0, seed=len(new) + 1)
    same = dict(d_n_free_out=c.d["n_free"].data_ptr())
    if ctx is not None:
        same["d_seq_len"] = c.d["ctx"].data_ptr()
    tok.paged_assign_device(c.args(**same))
    c.check(n_free="n_free", seq="seq" if ctx is None else "ctx")
    c = _Call(torch, pkg, new, ctx, bs, seed=5)
    tok.paged_assign_device(c.args(d_pos=None, d_req=None, d_seq_len=None))
    want = _expected(c.new, c.ctx, bs, c.table, c.free, c.n_free, c.cap)
    assert np.array_equal(c.host("slot")[:c.cap], want[1]) and np.array_equal(c.host("table"), want[0])
    assert (c.host("pos") == -9).all() and (c.host("req") == -9).all()


def test_assign_in_place_repeats(env):
    # a decode loop that only keeps its own buffers: each step starts where the last one ended
    torch, pkg, tok = env
    n, bs, steps = 1500, 4, 9
    ctx = np.random.default_rng(3).integers(0, 50, n).tolist()
    c = _Call(torch, pkg, [1] * n, ctx, bs, max_blocks=16, spare=n * 3)
    table, n_free = c.table, c.n_free
    for _ in range(steps):
        tok.paged_assign_device(c.args(d_n_free_out=c.d["n_free"].data_ptr(), d_seq_len=c.d["ctx"].data_ptr()))
        table, slot, pos, _, ctx, n_free = _expected([1] * n, ctx, bs, table, c.free, n_free, c.cap)
        assert np.array_equal(c.host("slot")[:c.cap], slot) and np.array_equal(c.host("pos")[:c.cap], pos)
    assert np.array_equal(c.host("table"), table) and c.host("n_free").tolist() == [n_free]
    assert np.array_equal(c.host("ctx"), ctx) and tok._L.tok_last_error(tok._h) is not None


@pytest.mark.parametrize("tokens,empty", [(128, 0), (256, 0), (512, 0), (128, 2), (512, 400), (1024, 4500)])
def test_assign_in_place_by_one_cta(env, tokens, empty):
    # one request brings all the tokens of a call that a single CTA takes, with no padding (a chunk of a
    # prefill), and its length is replaced by the same CTA
    torch, pkg, tok = env
    for seed in range(20):
        new, ctx = [0] * empty + [tokens] + [0] * empty, [1] * empty + [17 + seed] + [5] * empty
        c = _Call(torch, pkg, new, ctx, 16, spare=0, pad=0, seed=seed)
        tok.paged_assign_device(c.args(d_n_free_out=c.d["n_free"].data_ptr(), d_seq_len=c.d["ctx"].data_ptr()))
        c.check(n_free="n_free", seq="ctx")


def test_in_place_right_after_the_load(env):
    # a handle's counter of finished CTAs is 0 for the first call, on a stream that does not wait for the default one
    torch, pkg, _ = env
    s = torch.cuda.Stream()
    busy = torch.zeros(1 << 26, device="cuda")
    n = 1500
    for seed in range(6):
        c = _Call(torch, pkg, [1] * n, [7] * n, 4, seed=seed)
        torch.cuda.synchronize()
        busy.add_(1.0)
        tok = pkg.Tokenizer.from_merges([], pkg.PATTERN_GPT2)
        tok.paged_assign_device(c.args(d_n_free_out=c.d["n_free"].data_ptr(), d_seq_len=c.d["ctx"].data_ptr()), s.cuda_stream)
        s.synchronize()
        c.check(n_free="n_free", seq="ctx")
        tok.close()


@pytest.mark.parametrize("n", [3, 2000])
def test_assign_refuses_on_the_device(env, n):
    torch, pkg, tok = env
    new, ctx = [2] * n, [3] * n
    call = lambda **k: _Call(torch, pkg, new, ctx, 4, **k)  # noqa: E731
    run = lambda c, **k: tok.paged_assign_device(c.args(**k))  # noqa: E731
    c = call(spare=0)
    c.n_free -= 1
    c.d["n_free"][0] -= 1
    run(c)
    assert c.check_refused(pkg.TOK_EBUF, -1)[1] == n  # one block too few
    c = call(cap=2 * n - 1)
    run(c)
    assert c.check_refused(pkg.TOK_EBUF, -1)[2] == 2 * n
    c = call(max_blocks=1)
    run(c)
    c.check_refused(pkg.TOK_EBUF, 0)
    c = call()
    c.d["ctx"][1] = c.ctx[1] = -1
    run(c)
    c.check_refused(pkg.TOK_EINVAL, 1)
    c = call()
    c.d["ctx"][1] = c.ctx[1] = 2**31 - 1
    run(c)
    c.check_refused(pkg.TOK_EINVAL, 1)
    c = call()
    c.d["off"][2] = 1  # decreasing
    run(c)
    c.check_refused(pkg.TOK_EINVAL, 1)
    c = call()
    c.d["off"][0] = 1
    run(c)
    c.check_refused(pkg.TOK_EINVAL, 0)
    c = call()
    c.d["n_free"][0] = c.n_free = -1
    run(c)
    c.check_refused(pkg.TOK_EINVAL, -1)
    # the handle goes on
    c = call()
    run(c)
    c.check()


def _release_expected(lens, done, bs, table, free, n_free):
    out = free.copy()
    for k, (m, d) in enumerate(zip(lens, done)):
        if d:
            b = _blocks(m, bs)
            out[n_free:n_free + b] = table[k, :b]
            n_free += b
    return out, n_free


@pytest.mark.parametrize("n,most,bs,share", [(1, 0, 4, 1.0), (1, 9, 4, 1.0), (5, 100, 1, 0.5), (300, 70, 16, 0.3),
                                             (700, 50, 3, 1.0), (2000, 900, 7, 0.1), (40, 20_000, 16, 0.0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_release(env, n, most, bs, share, in_place):
    torch, pkg, tok = env
    rng = np.random.default_rng(n + most)
    lens, done = rng.integers(0, most + 1, n), (rng.random(n) < share).astype(np.uint8) * rng.integers(1, 256, n).astype(np.uint8)
    cols = max(1, _blocks(most, bs))
    table = rng.integers(0, 1 << 30, (n, cols + 2)).astype(np.int32)
    total = sum(_blocks(m, bs) for m, d in zip(lens, done) if d)
    free = np.full(10 + total + 2, -9, dtype=np.int32)
    free[:10] = np.arange(10)
    d = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in (
        ("lens", lens.astype(np.int64)), ("done", done), ("table", table), ("free", free),
        ("n_free", np.array([10])), ("out", np.array([-7])), ("status", np.full(4, -7)))}
    call = lambda cap: tok.paged_release_device(  # noqa: E731
        d["lens"].data_ptr(), d["done"].data_ptr(), n, bs, d["table"].data_ptr(), cols + 2, cols, d["free"].data_ptr(), cap,
        d["n_free"].data_ptr(), d["n_free" if in_place else "out"].data_ptr(), d["status"].data_ptr())
    if total:
        call(10 + total - 1)  # one entry too few: nothing happens
        assert d["status"].cpu().tolist() == [pkg.TOK_EBUF, total, 0, -1]
        assert np.array_equal(d["free"].cpu().numpy(), free)
        assert d["n_free" if in_place else "out"].cpu().tolist() == [10]
    call(10 + total)
    want, left = _release_expected(lens, done, bs, table, free, 10)
    assert d["status"].cpu().tolist() == [0, total, 0, -1]
    assert np.array_equal(d["free"].cpu().numpy(), want)
    assert d["n_free" if in_place else "out"].cpu().tolist() == [left]
    assert np.array_equal(d["table"].cpu().numpy(), table)
    # a length beyond the row, a negative one: refused with the first such request
    if n > 2:
        d["n_free"].fill_(10)
        d["done"][:] = 1
        d["lens"][:] = 0
        d["lens"][n - 1] = cols * bs + 1
        d["lens"][1] = -1
        call(10 + total)
        assert d["status"].cpu().tolist() == [pkg.TOK_EINVAL, 0, 0, 1]
        assert d["n_free" if in_place else "out"].cpu().tolist() == [10]


@pytest.mark.parametrize("n", [3, 2000])
def test_bad_numbers_count_no_blocks(env, n):
    # status[1] is what was taken or returned, and what is lacking only where that is the error
    torch, pkg, tok = env
    c = _Call(torch, pkg, [2] * n, [3] * n, 4)
    c.d["ctx"][1] = c.ctx[1] = -1
    tok.paged_assign_device(c.args())
    assert c.check_refused(pkg.TOK_EINVAL, 1)[1] == 0
    d = {k: torch.full((m,), v, dtype=t, device="cuda") for k, m, v, t in (
        ("lens", n, 5, torch.int64), ("done", n, 1, torch.uint8), ("free", 4 * n, -9, torch.int32), ("n_free", 1, 0, torch.int64),
        ("out", 1, -7, torch.int64), ("status", 4, -7, torch.int64))}
    d["lens"][2] = -1
    tok.paged_release_device(d["lens"].data_ptr(), d["done"].data_ptr(), n, 4, c.d["table"].data_ptr(), c.table.shape[1],
                             c.max_blocks, d["free"].data_ptr(), 4 * n, d["n_free"].data_ptr(), d["out"].data_ptr(),
                             d["status"].data_ptr())
    assert d["status"].cpu().tolist() == [pkg.TOK_EINVAL, 0, 0, 2]
    assert d["out"].cpu().tolist() == [0] and bool((d["free"] == -9).all())


def test_refusals_on_the_host(env):
    torch, pkg, tok = env
    c = _Call(torch, pkg, [2, 3], [1, 1], 4)
    for bad in (dict(d_item_off=None), dict(d_table=None), dict(d_free=None), dict(d_n_free=None), dict(d_n_free_out=None),
                dict(d_slot=None), dict(d_status=None), dict(n=0), dict(block_size=0), dict(block_size=(1 << 20) + 1),
                dict(table_stride=c.max_blocks - 1)):
        with pytest.raises(pkg.TokError) as e:
            tok.paged_assign_device(c.args(**bad))
        assert e.value.code == pkg.TOK_EINVAL and "paged assign" in str(e.value), bad
    assert tok._L.tok_paged_assign(None, c.args()._addr, None) == pkg.TOK_EINVAL
    assert tok._L.tok_paged_assign(tok._h, None, None) == pkg.TOK_EINVAL
    assert (c.host("slot") == -9).all()
    with pytest.raises(TypeError):
        pkg.PagedArgs(no_such_field=1)
    one = torch.ones(4, dtype=torch.int64, device="cuda")
    good = [one.data_ptr(), one.data_ptr(), 1, 4, one.data_ptr(), 2, 2, one.data_ptr(), 2, one.data_ptr(), one.data_ptr(), one.data_ptr()]
    for at, v in ((0, None), (1, None), (2, 0), (3, 0), (4, None), (5, 1), (7, None), (9, None), (10, None), (11, None)):
        bad = list(good)
        bad[at] = v
        with pytest.raises(pkg.TokError) as e:
            tok.paged_release_device(*bad)
        assert e.value.code == pkg.TOK_EINVAL and "paged release" in str(e.value), at


def test_device_batch_to_slots_in_a_graph(env):
    # the offsets of tok_encode_batch_device go straight in; captured once, replayed on another batch
    torch, pkg, tok = env
    texts = [b"hello world", b"", b"a" * 50]
    blob = b"".join(texts)
    n, cap, bs = len(texts), 256, 4
    start = torch.tensor(np.concatenate([[0], np.cumsum([len(t) for t in texts])]), dtype=torch.int64, device="cuda")
    text = torch.frombuffer(bytearray(blob), dtype=torch.uint8).cuda()
    ids, st = torch.empty(cap, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    c = _Call(torch, pkg, [0] * n, [3, 4, 0], bs, max_blocks=40, spare=100, cap=cap)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        tok.encode_batch_device(text.data_ptr(), len(blob), start.data_ptr(), n, ids.data_ptr(), cap, c.d["off"].data_ptr(),
                                st.data_ptr(), s.cuda_stream)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tok.paged_assign_device(c.args(), torch.cuda.current_stream().cuda_stream)
    for new in ([11, 0, 50], [1, 2, 3]):  # (one byte, one token)
        c.d["off"].copy_(torch.tensor(np.concatenate([[0], np.cumsum(new)])))
        c.d["table"].copy_(torch.from_numpy(c.table))
        g.replay()
        torch.cuda.synchronize()
        c.new, c.total = new, sum(new)
        c.taken = sum(_blocks(x + m, bs) - _blocks(x, bs) for x, m in zip(c.ctx, new))
        c.check()
    assert st.cpu().tolist()[:2] == [0, 61] and isinstance(tok.launch_count, int) and ctypes
