"""tok_paged_store and tok_paged_attend against plain loops in 64 bits: lengths
from nothing to long ones, block sizes of 1 and odd ones, groups and widths that
do not fill a tile, layouts, windows, tables with entries that name no block,
and the refusals."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

KINDS = ["f16", "bf16"]


@pytest.fixture(scope="module")
def env():
    import torch

    from exact_bpe_tokenization_utf_gb300 import _build
    _build.build()
    import exact_bpe_tokenization_utf_gb300 as pkg
    tok = pkg.Tokenizer.from_merges([], pkg.PATTERN_GPT2)
    yield torch, pkg, tok
    tok.close()


class _Cache:
    """Keys and values [block, place, head, width] in one of the layouts, with a struct."""

    def __init__(self, env, kind, n_blocks, bs, heads, dim, layout="token", seed=0, gap=0):
        torch, pkg, _ = env
        self.torch, self.pkg = torch, pkg
        self.dtype = {"f16": torch.float16, "bf16": torch.bfloat16}[kind]
        self.bs, self.heads, self.dim, self.n_blocks = bs, heads, dim, n_blocks
        g = torch.Generator(device="cuda").manual_seed(seed)
        size = (n_blocks, bs, heads, dim + gap) if layout == "token" else (n_blocks, heads, bs, dim + gap)
        both = [torch.randn(*size, generator=g, device="cuda").to(self.dtype) for _ in range(2)]
        self.k, self.v = [(t if layout == "token" else t.transpose(1, 2))[..., :dim] for t in both]
        self.kind = kind

    def struct(self, **other):
        f = dict(d_k=self.k.data_ptr(), d_v=self.v.data_ptr(), block_stride=self.k.stride(0), token_stride=self.k.stride(1),
                 head_stride=self.k.stride(2), dtype=self.pkg.DTYPE_F16 if self.kind == "f16" else self.pkg.DTYPE_BF16,
                 n_blocks=self.n_blocks, block_size=self.bs, kv_heads=self.heads, head_dim=self.dim)
        f.update(other)
        return self.pkg.KVCache(**f)


class _Attend:
    def __init__(self, env, lens, group, cache, window=0, scale=None, seed=1, spare=2, q_size=1.0):
        self.torch, self.pkg, self.tok = env
        torch = self.torch
        self.cache, self.window, self.lens = cache, window, [int(x) for x in lens]
        self.n, self.heads = len(lens), cache.heads * group
        self.scale = cache.dim ** -0.5 if scale is None else scale
        rng = np.random.default_rng(seed)
        need = [-(-max(m, 0) // cache.bs) for m in self.lens]
        self.max_blocks = max(need + [1])
        table = np.full((self.n, self.max_blocks + spare), -1, np.int32)
        order = rng.permutation(cache.n_blocks)
        at = 0
        for r, m in enumerate(need):
            table[r, :m] = order[np.arange(at, at + m) % cache.n_blocks]   # (requests may share blocks)
            at += m
        table[:, self.max_blocks:] = 1 << 30   # behind the row: never used
        self.table = torch.from_numpy(table).cuda()
        self.seq_len = torch.tensor(self.lens, dtype=torch.int64, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q = (torch.randn(self.n, self.heads, cache.dim, generator=g, device="cuda") * q_size).to(cache.dtype)
        self.out = torch.full((self.n + 1, self.heads, cache.dim), 7.0, dtype=cache.dtype, device="cuda")
        self.lse = torch.full((self.n + 1, self.heads), 7.0, device="cuda")
        size = self.tok.attend_work_bytes(self.n, self.heads, cache.heads, cache.dim)
        self.work = torch.full((size,), 0xee, dtype=torch.uint8, device="cuda")

    def run(self, cache=None, **other):
        D = self.cache.dim
        f = dict(d_q=self.q.data_ptr(), q_stride=self.q.stride(0), q_head_stride=self.q.stride(1), d_out=self.out.data_ptr(),
                 out_stride=self.heads * D, out_head_stride=D, d_lse=self.lse.data_ptr(), n=self.n, heads=self.heads,
                 scale=self.scale, window=self.window, d_table=self.table.data_ptr(), table_stride=self.table.stride(0),
                 max_blocks=self.max_blocks, d_seq_len=self.seq_len.data_ptr(), d_work=self.work.data_ptr(),
                 work_bytes=self.work.numel())
        f.update(other)
        self.tok.paged_attend_device(cache or self.cache.struct(), self.pkg.AttendArgs(**f),
                                     self.torch.cuda.current_stream().cuda_stream)

    def want(self):
        """(out, lse, sum of weight times size of the values) in 64 bits, by request and key head."""
        torch, c = self.torch, self.cache
        out = torch.zeros(self.n, self.heads, c.dim, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(out)
        lse = torch.full((self.n, self.heads), -math.inf, dtype=torch.float64, device="cuda")
        group = self.heads // c.heads
        scale = float(np.float32(self.scale))
        for r, m in enumerate(self.lens):
            m = min(max(m, 0), self.max_blocks * c.bs)
            p = torch.arange(max(0, m - self.window) if self.window else 0, m, device="cuda")
            block = self.table[r, (p // c.bs)].long()
            ok = (block >= 0) & (block < c.n_blocks)
            p, block = p[ok], block[ok]
            if not len(p):
                continue
            for h in range(c.heads):
                k, v = (t[block, p % c.bs, h].double() for t in (c.k, c.v))
                j = slice(h * group, (h + 1) * group)
                s = self.q[r, j].double() @ k.t() * scale
                w = torch.softmax(s, 1)
                out[r, j], size[r, j], lse[r, j] = w @ v, w @ v.abs(), torch.logsumexp(s, 1)
        return out, lse, size

    def check(self, run=True):
        torch = self.torch
        if run:
            self.run()
        out, lse, size = self.want()
        got, got_lse = self.out[:self.n].double(), self.lse[:self.n].double()
        # scores: products exact, D + 4 roundings of 32 bits on sums no larger than the row's largest sum of
        # sizes, the product with the scale and the exponential's argument; a weight is off by as much, and by
        # 2^-16 (two 16-bit numbers) or 2^-22 (the exponential); sums of weights add a rounding for each of the
        # tokens in a thread's chain, far fewer than 2^10; then the type's rounding
        big = max(1.0, float(self.q.double().abs().sum(2).max()) * float(self.cache.k.double().abs().max()) * abs(self.scale))
        off = big * (self.cache.dim + 4) * 2.0**-24 + 2.0**-16 + 2.0**-14
        half = torch.finfo(self.cache.dtype).eps / 2
        tol = size * off * 2 + out.abs() * half * (1 + 2.0**-8) + 2.0**-25
        assert bool(((got - out).abs() <= tol).all()), float(((got - out).abs() - tol).max())
        empty = lse == -math.inf
        assert bool((got_lse[empty] == -math.inf).all()) and bool((got[empty] == 0).all())
        assert bool(((got_lse - lse).abs()[~empty] <= off + lse.abs()[~empty] * 2.0**-22).all())
        assert bool((self.out[self.n:] == 7).all()) and bool((self.lse[self.n:] == 7).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [8, 16, 40, 64, 72, 80, 128, 136, 192, 256])
def test_widths_and_groups(env, kind, dim):
    for heads, group in ((1, 1), (2, 3), (3, 8), (2, 9), (1, 16), (1, 17), (1, 64)):
        c = _Cache(env, kind, 40, 16, heads, dim, layout="head" if group % 2 else "token", seed=dim, gap=8 if heads == 2 else 0)
        _Attend(env, [100, 1, 0, 333, 64], group, c, seed=group).check()


@pytest.mark.parametrize("bs", [1, 2, 7, 16, 33, 48, 64, 129, 1000])
def test_blocks(env, bs):
    lens = [0, 1, 2, bs - 1, bs, bs + 1, 15, 16, 17, 63, 64, 65, 127, 500, 1025, 3 * bs]
    c = _Cache(env, "bf16", -(-sum(lens) // bs) + 20, bs, 2, 64, seed=bs)
    _Attend(env, lens, 4, c).check()
    _Attend(env, lens[::-1], 4, c, window=37).check()


@pytest.mark.parametrize("kind", KINDS)
def test_long_and_short_requests_together(env, kind):
    c = _Cache(env, kind, 3000, 16, 2, 128, layout="head")
    _Attend(env, [40001, 3, 0, 0, 1, 700, 0, 20000, 64], 8, c).check()
    _Attend(env, [30011], 5, c).check()
    _Attend(env, [0, 0, 0], 5, c).check()
    _Attend(env, [5] * 700, 2, c).check()
    _Attend(env, list(range(0, 400)), 1, c).check()


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 1000, 4096, 1 << 31])
def test_windows(env, window):
    c = _Cache(env, "bf16", 500, 24, 1, 64)
    _Attend(env, [0, 1, 2, 16, 17, 63, 100, 999, 1000, 1001, 6000], 8, c, window=window).check()


def test_entries_that_name_no_block(env):
    torch = env[0]
    c = _Cache(env, "f16", 60, 16, 2, 64)
    a = _Attend(env, [200, 16, 17, 320, 48], 4, c)
    a.table[0, 3] = -1
    a.table[0, 7] = 60
    a.table[1, 0] = 1 << 30
    a.table[2, 1] = -5
    a.table[3, ::2] = -1
    a.table[4, :] = -(1 << 31)
    a.check()
    # NaN in blocks that nothing names, and behind the last token of a block, has no influence
    used = torch.unique(a.table[:, :a.max_blocks])
    unused = [b for b in range(60) if b not in set(used.tolist())]
    c.k[unused], c.v[unused] = float("nan"), float("inf")
    b = a.table[2, 0].item()
    a.check()
    one = _Attend(env, [5], 4, c, seed=3)
    one.table[0, 0] = b
    keep = c.k[b, 5:].clone(), c.v[b, 5:].clone()
    c.k[b, 5:], c.v[b, 5:] = float("nan"), float("inf")
    one.check()
    c.k[b, 5:], c.v[b, 5:] = keep


def test_lengths_that_make_no_sense(env):
    torch = env[0]
    c = _Cache(env, "bf16", 60, 8, 1, 64)
    a = _Attend(env, [30, 64, 9], 4, c)
    a.lens = [30, -7, 10**12]
    a.table[2, :a.max_blocks] = torch.arange(a.max_blocks, dtype=torch.int32, device="cuda")
    a.seq_len.copy_(torch.tensor(a.lens))
    a.check()


@pytest.mark.parametrize("kind", KINDS)
def test_steep_and_flat_scores(env, kind):
    torch = env[0]
    c = _Cache(env, kind, 200, 16, 2, 64)
    for scale, size in ((1.0, 30.0), (0.0, 1.0), (-0.5, 1.0), (50.0, 1.0), (1e-4, 1.0)):
        a = _Attend(env, [1000, 77, 500], 4, c, scale=scale, q_size=size)
        a.run()
        out, lse, _ = a.want()
        # scores of some thousands: their 32-bit rounding moves the weights
        s = float(np.abs(scale)) * float(a.q.double().abs().sum(2).max()) * float(c.k.double().abs().max())
        off = max(1.0, s) * 70 * 2.0**-24
        assert bool(torch.isfinite(a.out[:3]).all())
        assert bool(((a.lse[:3].double() - lse).abs() <= off + 2.0**-13 + lse.abs() * 2.0**-22).all())
        if off < 0.01:
            a.check(run=False)
    # scores that rise all along: the reference is replaced again and again
    k = torch.linspace(-40, 40, 160 * 16, device="cuda").view(160, 16)
    c.k[:160, :, :, 0] = k[:, :, None].to(c.k.dtype)
    a = _Attend(env, [2500], 4, c, scale=1.0, q_size=0.01)
    a.table[0, :160] = torch.arange(160, dtype=torch.int32, device="cuda")[:a.table.shape[1]]
    a.q[:, :, 0] = 4.0
    a.check()
    a.q[:, :, 0] = -4.0
    a.check()


def test_infinite_values_and_scores(env):
    torch = env[0]
    c = _Cache(env, "bf16", 20, 16, 1, 64)
    a = _Attend(env, [40, 40], 2, c)
    b = a.table[0, 0].item()
    c.v[b, 3, 0, 5] = float("inf")
    a.run()
    assert bool((a.out[0, :, 5] == float("inf")).all())
    a2 = _Attend(env, [40], 2, c)
    a2.table[0] = a.table[0, :a2.table.shape[1]]
    c.k[b, 3, 0, 0] = float("nan")
    a2.run()
    assert bool(torch.isnan(a2.out[0]).all()) and bool(torch.isnan(a2.lse[0]).all())


def test_many_requests(env):
    rng = np.random.default_rng(0)
    c = _Cache(env, "bf16", 600, 4, 1, 8)
    _Attend(env, rng.integers(0, 30, 5000), 1, c).check()


def test_offsets_beyond_32_bits(env):
    # a cache of more than 2^32 elements, whose last blocks are read and written
    torch, pkg, tok = env
    n_blocks, bs, heads, dim = 17000, 16, 64, 256
    k = torch.zeros(n_blocks, bs, heads, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(1)
    small = _Cache(env, "bf16", 4, bs, heads, dim)
    big = _Cache.__new__(_Cache)
    big.__dict__.update(small.__dict__)
    big.k, big.v, big.n_blocks = k, v, n_blocks
    new = torch.randn(2 * bs, 2 * heads, dim, generator=g, device="cuda").bfloat16()
    slot = torch.cat([torch.arange(bs) + (n_blocks - 1) * bs, torch.arange(bs) + (n_blocks - 300) * bs]).cuda()
    tok.paged_store_device(big.struct(), pkg.StoreArgs(d_k=new.data_ptr(), d_v=new[:, heads:].data_ptr(), token_stride=new.stride(0),
                                                       head_stride=new.stride(1), d_slot=slot.data_ptr(), n=2 * bs))
    torch.cuda.synchronize()
    assert torch.equal(k[-1], new[:bs, :heads]) and torch.equal(v[n_blocks - 300], new[bs:, heads:])
    a = _Attend(env, [30], 1, big)
    a.table[0, 0], a.table[0, 1] = n_blocks - 1, n_blocks - 300
    a.run()
    small.k[0], small.v[0], small.k[1], small.v[1] = k[-1], v[-1], k[n_blocks - 300], v[n_blocks - 300]
    b = _Attend(env, [30], 1, small)
    b.table[0, 0], b.table[0, 1] = 0, 1
    b.q.copy_(a.q)
    b.check()
    assert torch.equal(a.out, b.out)


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("kind", KINDS)
def test_store(env, kind, layout):
    torch, pkg, tok = env
    for n, heads, dim, bs in ((1, 1, 8, 1), (33, 2, 64, 16), (500, 3, 80, 7), (1000, 8, 128, 33), (40, 1, 256, 16)):
        c = _Cache(env, kind, -(-n // bs) + 9, bs, heads, dim, layout=layout, gap=8)
        k0, v0 = c.k.clone(), c.v.clone()
        new = torch.randn(n, 2 * heads + 1, dim, device="cuda").to(c.dtype)
        slot = torch.randperm(c.n_blocks * bs, device="cuda")[:n]
        slot[torch.rand(n, device="cuda") < 0.2] = -1
        slot[: n // 9] = c.n_blocks * bs + torch.arange(n // 9, device="cuda")
        if n > 20:
            slot[n - 1], slot[n - 2] = 1 << 62, -(1 << 62)
        args = pkg.StoreArgs(d_k=new.data_ptr(), d_v=new[:, heads:].data_ptr(), token_stride=new.stride(0),
                             head_stride=new.stride(1), d_slot=slot.data_ptr(), n=n)
        tok.paged_store_device(c.struct(), args)
        ok = (slot >= 0) & (slot < c.n_blocks * bs)
        k0[slot[ok] // bs, slot[ok] % bs] = new[ok][:, :heads]
        v0[slot[ok] // bs, slot[ok] % bs] = new[ok][:, heads:2 * heads]
        assert torch.equal(c.k, k0) and torch.equal(c.v, v0)


def test_a_prompt_and_steps_through_the_cache(env):
    """assign, store and attend as a decoder uses them: every step's attention is that over the keys so far."""
    torch, pkg, tok = env
    n, heads, group, dim, bs = 5, 2, 4, 64, 16
    prompts = np.array([40, 1, 0, 17, 100])
    steps = 20
    c = _Cache(env, "bf16", 60, bs, heads, dim)
    max_blocks = -(-(int(prompts.max()) + steps) // bs)
    table = torch.full((n, max_blocks), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(60, device="cuda").to(torch.int32)
    n_free = torch.tensor([60], device="cuda")
    seq = torch.zeros(n, dtype=torch.int64, device="cuda")
    status = torch.zeros(4, dtype=torch.int64, device="cuda")
    history = [[] for _ in range(n)]
    for step in range(steps):
        new = prompts if step == 0 else np.ones(n, int)
        total = int(new.sum())
        off = torch.tensor(np.concatenate([[0], np.cumsum(new)]), device="cuda")
        cap = total + 3   # a padded batch
        slot = torch.empty(cap, dtype=torch.int64, device="cuda")
        tok.paged_assign_device(pkg.PagedArgs(
            d_item_off=off.data_ptr(), d_ctx_len=seq.data_ptr(), n=n, block_size=bs, d_table=table.data_ptr(),
            table_stride=max_blocks, max_blocks=max_blocks, d_free=free.data_ptr(), d_n_free=n_free.data_ptr(),
            d_n_free_out=n_free.data_ptr(), d_slot=slot.data_ptr(), cap=cap, d_seq_len=seq.data_ptr(), d_status=status.data_ptr()))
        kv = torch.randn(cap, 2 * heads, dim, device="cuda").bfloat16()
        tok.paged_store_device(c.struct(), pkg.StoreArgs(d_k=kv.data_ptr(), d_v=kv[:, heads:].data_ptr(), token_stride=kv.stride(0),
                                                         head_stride=dim, d_slot=slot.data_ptr(), n=cap))
        at = 0
        for r in range(n):
            history[r].append(kv[at:at + new[r]])
            at += new[r]
        a = _Attend.__new__(_Attend)
        a.torch, a.pkg, a.tok, a.cache, a.window, a.n, a.heads, a.scale = torch, pkg, tok, c, 0, n, heads * group, dim ** -0.5
        a.table, a.seq_len, a.max_blocks = table, seq, max_blocks
        a.lens = seq.tolist()
        assert a.lens == [int(p) + step for p in prompts]
        a.q = torch.randn(n, heads * group, dim, device="cuda").bfloat16()
        a.out = torch.full((n + 1, heads * group, dim), 7.0, dtype=torch.bfloat16, device="cuda")
        a.lse = torch.full((n + 1, heads * group), 7.0, device="cuda")
        a.work = torch.empty(tok.attend_work_bytes(n, heads * group, heads, dim), dtype=torch.uint8, device="cuda")
        a.check()
        if step == steps - 1:
            for r in range(n):
                h = torch.cat(history[r])
                p = torch.arange(len(h), device="cuda")
                assert torch.equal(c.k[table[r, p // bs].long(), p % bs], h[:, :heads])


def test_the_same_bits_each_time_and_graphs(env):
    torch, pkg, tok = env
    c = _Cache(env, "bf16", 400, 16, 2, 128)
    a = _Attend(env, [3000, 5, 700, 1200], 8, c)
    a.check()
    want, want_lse = a.out.clone(), a.lse.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a.run()
    side.synchronize()
    assert torch.equal(a.out, want)
    works = [torch.empty_like(a.work) for _ in range(2)]
    outs = [torch.empty_like(a.out) for _ in range(2)]
    graphs = []
    for w, o in zip(works, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a.run(d_work=w.data_ptr(), d_out=o.data_ptr(), d_lse=None)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[:4], want[:4]) for o in outs)
    assert torch.equal(a.lse, want_lse)


def test_refusals(env):
    torch, pkg, tok = env
    c = _Cache(env, "bf16", 10, 16, 2, 64)
    a = _Attend(env, [20, 30], 4, c)
    for other in (dict(d_k=None), dict(d_v=None), dict(dtype=pkg.DTYPE_F32), dict(dtype=9), dict(n_blocks=0), dict(block_size=0),
                  dict(block_size=(1 << 20) + 1), dict(kv_heads=0), dict(kv_heads=1025), dict(kv_heads=3), dict(head_dim=0),
                  dict(head_dim=60), dict(head_dim=264), dict(token_stride=68), dict(head_stride=-64), dict(block_stride=4),
                  dict(d_k=c.k.data_ptr() + 8)):
        with pytest.raises(pkg.TokError) as e:
            a.run(cache=c.struct(**other))
        assert e.value.code == pkg.TOK_EINVAL, other
    for other in (dict(d_q=None), dict(d_out=None), dict(d_table=None), dict(d_seq_len=None), dict(d_work=None), dict(work_bytes=64),
                  dict(heads=0), dict(heads=7), dict(heads=2 * 65), dict(n=(1 << 20) + 1), dict(table_stride=1, max_blocks=2),
                  dict(max_blocks=1 << 31), dict(q_stride=4), dict(q_head_stride=1), dict(out_stride=2), dict(out_head_stride=3),
                  dict(d_q=a.q.data_ptr() + 2), dict(d_out=a.out.data_ptr() + 8), dict(d_work=a.work.data_ptr() + 16),
                  dict(d_lse=a.lse.data_ptr() + 1), dict(d_seq_len=a.seq_len.data_ptr() + 4)):
        with pytest.raises(pkg.TokError) as e:
            a.run(**other)
        assert e.value.code == pkg.TOK_EINVAL, other
    new = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    slot = torch.zeros(4, dtype=torch.int64, device="cuda")
    good = dict(d_k=new.data_ptr(), d_v=new.data_ptr(), token_stride=256, head_stride=64, d_slot=slot.data_ptr(), n=4)
    for other in (dict(d_k=None), dict(d_v=None), dict(d_slot=None), dict(token_stride=4), dict(head_stride=1), dict(n=1 << 31),
                  dict(d_k=new.data_ptr() + 2), dict(d_slot=slot.data_ptr() + 4)):
        with pytest.raises(pkg.TokError) as e:
            tok.paged_store_device(c.struct(), pkg.StoreArgs(**dict(good, **other)))
        assert e.value.code == pkg.TOK_EINVAL, other
    a.run(n=0, d_q=None, d_out=None, d_work=None)
    tok.paged_store_device(c.struct(), pkg.StoreArgs(**dict(good, n=0, d_k=None)))
    torch.cuda.synchronize()
    assert bool((a.out == 7).all())
    assert tok.attend_work_bytes(1, 7, 2, 64) == 0 and tok.attend_work_bytes(1, 8, 2, 60) == 0
    assert tok.attend_work_bytes(4, 8, 2, 64) <= tok.attend_work_bytes(5, 8, 2, 64)


def _in_a_row(env, cache, lens, group=1, **other):
    """An _Attend whose requests have the cache's blocks one after another."""
    a = _Attend(env, lens, group, cache, spare=0, **other)
    a.table.fill_(-1)
    at = 0
    for r, m in enumerate(lens):
        need = -(-m // cache.bs)
        a.table[r, :need] = env[0].arange(at, at + need, dtype=env[0].int32, device="cuda")
        at += need
    assert at <= cache.n_blocks
    return a


@pytest.mark.parametrize("kind", KINDS)
def test_weights_keep_their_bits(env, kind):
    # Values that the weights make cancel: what is left of out is far below its terms, so that a weight's error
    # shows.  A token of score 0 and value 0, then four of scores in -1 .. 0, each of whose values takes away
    # what the ones before leave.
    torch = env[0]
    n, heads, dim = 40, 8, 64
    c = _Cache(env, kind, n, 5, heads, dim)
    g = torch.Generator(device="cuda").manual_seed(2)
    s = -torch.randint(1, 128, (n, 5, heads), generator=g, device="cuda").double() / 128
    s[:, 0] = 0
    c.k.zero_()
    c.k[..., 0] = s
    w = s.exp()[..., None]
    v = torch.zeros(n, 5, heads, dim, dtype=torch.float64, device="cuda")
    v[:, 1] = 1 + torch.rand(n, heads, dim, generator=g, device="cuda").to(c.dtype).double()
    v[:, 1] = v[:, 1].to(c.dtype).double()
    for t in range(2, 5):
        v[:, t] = (-(w * v).sum(1) / w[:, t]).to(c.dtype).double()
    c.v.copy_(v)
    a = _in_a_row(env, c, [5] * n, scale=1.0)
    a.q.zero_()
    a.q[..., 0] = 1
    a.run()
    out, lse, size = a.want()
    # A score is exact; its product with log2(e) and the reference's are off by 2 roundings of at most 1.45 each,
    # their difference by one more: 2^-21.2 in all, times ln 2.  The exponential: 2^-22.  A weight's parts: 2^-22.
    # Sums of 5 tokens' products in 2 or 3 parts: a product of matrices adds each part to within 2^-22 of its
    # terms, 2^-20.4.  The sum of weights and the quotient: 2^-22 of out, which is small.
    half = torch.finfo(c.dtype).eps / 2
    tol = size * 2.0**-19 + out.abs() * half * (1 + 2.0**-8) + 2.0**-25
    assert float(out.abs().max()) < float(size.min()) * 2.0**-15
    assert bool(((a.out[:n].double() - out).abs() <= tol).all()), float(((a.out[:n].double() - out).abs() / size).max()) * 2.0**19
    assert bool(((a.lse[:n].double() - lse).abs() <= 2.0**-19).all())


@pytest.mark.parametrize("depth", [9.0, 12.0, 14.0, 16.0, 17.6, 20.0, 26.0])
@pytest.mark.parametrize("kind", KINDS)
def test_small_weights_count(env, kind, depth):
    # A first token that takes nearly the whole weight and whose value is 0: out is what the others' small weights
    # make of theirs.  So many requests that a CTA has most of a request's tokens beside that one.
    torch, pkg, tok = env
    n, m, dim = 330, 4096, 64
    c = _Cache(env, kind, m // 16, 16, 2, dim, seed=3)
    g = torch.Generator(device="cuda").manual_seed(7)
    c.k.zero_()
    c.k[..., 0] = (-depth + (torch.rand(m // 16, 16, 2, generator=g, device="cuda") - 0.5) / 2).to(c.dtype)
    c.v[:, :, 1] = 1   # (one key head's values have no sign to cancel by)
    c.k[0, 0], c.v[0, 0] = 0, 0
    a = _in_a_row(env, c, [m], scale=1.0)
    a.q.zero_()
    a.q[..., 0] = 1
    out, lse, size = a.want()
    many = _Attend(env, [m] * n, 1, c, scale=1.0)
    many.table[:, :a.table.shape[1]] = a.table
    many.q.copy_(a.q.expand(n, -1, -1))
    many.want = lambda: tuple(t.expand(n, *t.shape[1:]) for t in (out, lse, size))
    many.check()


def _put(c, a, r, p, head, d, x):
    c.v[a.table[r, p // c.bs].long(), p % c.bs, head, d] = x


@pytest.mark.parametrize("q_size", [1.0, 40.0])
@pytest.mark.parametrize("dim,group", [(64, 8), (128, 16), (256, 3), (40, 1)])
@pytest.mark.parametrize("kind", KINDS)
def test_infinities_among_the_values(env, kind, dim, group, q_size):
    # every weight is above 0, however small: an infinity is out's, two of both signs and a NaN make a NaN
    torch = env[0]
    inf = float("inf")
    for seed in range(4):
        rng = np.random.default_rng(seed)
        lens = [1, 1, 2, 40, 17, 333, 0, 20011, 1000]
        c = _Cache(env, kind, 1500, 16, 2, dim, layout="head" if seed % 2 else "token", seed=seed)
        a = _in_a_row(env, c, lens, group=group, seed=seed, q_size=q_size)
        a.window = 700 if seed == 3 else 0
        out, lse, size = a.want()
        for r, m in enumerate(lens):
            for _ in range(12 if m else 0):
                p, h, d, x = int(rng.integers(m)), int(rng.integers(2)), int(rng.integers(dim)), float(rng.choice([inf, -inf, inf, -inf, np.nan]))
                _put(c, a, r, p, h, d, x)
        # (what the queries read, as the caches have it now: later ones replaced some)
        group_of = a.heads // c.heads
        special = torch.zeros_like(out)
        for r, m in enumerate(lens):
            p = torch.arange(max(0, m - a.window) if a.window else 0, m, device="cuda")
            v = c.v[a.table[r, p // c.bs].long(), p % c.bs].double()
            both = torch.where(torch.isfinite(v), 0.0, v).sum(0)          # inf, -inf, NaN or 0 for each key head and column
            special[r] = both.repeat_interleave(group_of, 0)
        a.run()
        got = a.out[:a.n].double()
        odd = special != 0   # (a NaN too)
        assert bool(odd.any())
        assert bool(torch.equal(torch.isnan(got), torch.isnan(special)))
        assert bool((got[odd] == special[odd])[~torch.isnan(special[odd])].all())
        assert bool(torch.isfinite(got[~odd]).all())
        if q_size == 1:
            # the others as ever
            off = max(1.0, float(a.q.double().abs().sum(2).max()) * float(c.k.double().abs().max()) * a.scale) * (dim + 4) * 2.0**-24 + 2.0**-13
            tol = torch.where(odd, 0.0, size * off * 2 + out.abs() * torch.finfo(c.dtype).eps / 2 * (1 + 2.0**-8) + 2.0**-25)
            assert bool(((torch.where(odd, 0.0, got) - torch.where(odd, 0.0, out)).abs() <= tol).all())
            assert bool(torch.isfinite(a.lse[:a.n][lse > -inf]).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,kv,group", [(64, 2, 4), (128, 2, 8), (80, 3, 5), (256, 1, 12), (64, 1, 20)])
def test_queries_and_outputs_with_strides(env, kind, dim, kv, group):
    # queries as slices of the rows of one product for queries, keys and values; outputs in wider rows, head by
    # head, and over the queries themselves
    torch = env[0]
    lens = [100, 1, 0, 5000, 64, 333]
    n, heads = len(lens), kv * group
    c = _Cache(env, kind, 400, 16, kv, dim)
    a = _Attend(env, lens, group, c)
    a.check()
    want, want_lse = a.out.clone(), a.lse.clone()
    wide = torch.full((n, heads + 2 * kv, dim + 8), float("nan"), dtype=c.dtype, device="cuda")
    wide[:, :heads, :dim] = a.q
    q = dict(d_q=wide.data_ptr(), q_stride=wide.stride(0), q_head_stride=wide.stride(1))

    def store(*size):
        return torch.full(size, 9.0, dtype=c.dtype, device="cuda")

    rows = store(n + 1, heads + 3, dim + 16)
    a.run(**q, d_out=rows[:, 1:].data_ptr(), out_stride=rows.stride(0), out_head_stride=rows.stride(1))
    assert torch.equal(rows[:n, 1:heads + 1, :dim], want[:n])
    rows[:n, 1:heads + 1, :dim] = 9
    assert bool((rows == 9).all())
    by_head = store(heads, n + 1, dim)
    a.lse.fill_(7)
    a.run(**q, d_out=by_head.data_ptr(), out_stride=by_head.stride(1), out_head_stride=by_head.stride(0))
    assert torch.equal(by_head[:, :n].transpose(0, 1), want[:n]) and bool((by_head[:, n] == 9).all())
    assert torch.equal(a.lse, want_lse)
    backwards = store(n, heads, dim)   # (strides below 0 are strides, too)
    a.run(**q, d_out=backwards[n - 1].data_ptr(), out_stride=-backwards.stride(0), out_head_stride=dim)
    assert torch.equal(backwards.flip(0), want[:n])
    over = a.q.clone()
    a.run(d_q=over.data_ptr(), d_out=over.data_ptr())
    assert torch.equal(over, want[:n])


@pytest.mark.parametrize("kind", KINDS)
def test_values_at_the_types_end(env, kind):
    # a mean of finite values is finite, and not above them
    torch = env[0]
    for dim, group in ((64, 8), (128, 12), (256, 2)):
        c = _Cache(env, kind, 1400, 16, 2, dim, seed=dim)
        most = torch.finfo(c.dtype).max
        c.v[:, :, 0] = most
        c.v[:, :, 1] = torch.where(c.v[:, :, 1] < 0, -most, most)
        lens = [1, 2, 40, 333, 20011]
        for q_size in (1.0, 20.0):
            a = _in_a_row(env, c, lens, group=group, seed=dim, q_size=q_size)
            a.run()
            got, half = a.out[:len(lens)].double(), torch.finfo(c.dtype).eps / 2
            assert bool(torch.isfinite(got).all())
            assert bool((got[:, :group] == most).all())
            if q_size == 1:
                out, lse, size = a.want()
                off = max(1.0, float(a.q.double().abs().sum(2).max()) * float(c.k.double().abs().max()) * a.scale) * (dim + 4) * 2.0**-24 + 2.0**-13
                assert bool(((got - out).abs() <= size * off * 2 + out.abs() * half * (1 + 2.0**-8)).all())
                assert bool(((a.lse[:len(lens)].double() - lse).abs() <= off + lse.abs() * 2.0**-22).all())
