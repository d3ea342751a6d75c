"""A decode loop through every operator at the model's two ends and at its cache:
ids become rows, keys and values go into the paged cache at the slots that
tok_paged_assign gave, the new tokens attend, the scores pass through
tok_logits_process, tok_sample chooses, and the choices are the next step's ids.
The step is captured in one graph; each of its results is compared with a plain
evaluation in 64 bits on what the step read.  At the end the gradient of the
embedding from all tokens of the run."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


class _Model:
    V, DIM, HEADS, KV, HEAD, BLOCK, STEPS = 1257, 128, 8, 2, 32, 16, 12

    def __init__(self, torch, pkg, tok, prompts):
        self.torch, self.pkg, self.tok, self.n = torch, pkg, tok, len(prompts)
        g = torch.Generator(device="cuda").manual_seed(3)
        n = self.n

        def weight(*size):
            return (torch.randn(*size, generator=g, device="cuda") / size[-1] ** 0.5).bfloat16()

        self.embed = weight(self.V, self.DIM)
        self.wq, self.wo = weight(self.HEADS * self.HEAD, self.DIM), weight(self.DIM, self.HEADS * self.HEAD)
        self.wkv, self.head = weight(2 * self.KV * self.HEAD, self.DIM), weight(self.V, self.DIM) * 6
        lens = [len(p) for p in prompts]
        self.max_blocks = -(-(max(lens) + self.STEPS) // self.BLOCK)
        self.n_blocks = n * self.max_blocks
        self.k, self.v = (torch.zeros(self.n_blocks, self.BLOCK, self.KV, self.HEAD, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.table = torch.full((n, self.max_blocks), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(self.n_blocks, generator=g, device="cuda").to(torch.int32)
        self.n_free = torch.tensor([self.n_blocks], device="cuda")
        self.seq = torch.zeros(n, dtype=torch.int64, device="cuda")
        self.status = torch.zeros(4, dtype=torch.int64, device="cuda")
        self.prompt = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device="cuda")
        self.prompt_off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device="cuda")
        self.one_off = torch.arange(n + 1, device="cuda")
        self.ids = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.random = torch.zeros(n, device="cuda")
        self.temperature = torch.full((n,), 0.8, device="cuda")
        self.top_p, self.top_k = torch.full((n,), 0.95, device="cuda"), torch.tensor([0, 40, 5, 0], dtype=torch.int32, device="cuda")[:n]
        self.logits = torch.zeros(n, self.V, dtype=torch.bfloat16, device="cuda")
        self.scores = torch.zeros_like(self.logits)
        self.kept = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.logprob = torch.zeros(n, device="cuda")
        self.out = torch.zeros(n, self.HEADS, self.HEAD, dtype=torch.bfloat16, device="cuda")
        self.work = torch.empty(tok.attend_work_bytes(n, self.HEADS, self.KV, self.HEAD), dtype=torch.uint8, device="cuda")
        self.keep = []

    def stream(self):
        return self.torch.cuda.current_stream().cuda_stream

    def rows(self, ids, off, cap):
        """Ids to rows, their keys and values into the cache; item off[k] .. off[k + 1] is request k's."""
        torch, pkg, tok = self.torch, self.pkg, self.tok
        x = torch.zeros(cap, self.DIM, dtype=torch.bfloat16, device="cuda")
        tok.embed_device(pkg.EmbedArgs(
            d_ids=ids.data_ptr(), n=cap, d_n=off[self.n:].data_ptr(), d_weight=self.embed.data_ptr(), weight_stride=self.DIM,
            weight_dtype=pkg.DTYPE_BF16, n_rows=self.V, dim=self.DIM, scale=self.DIM ** 0.5, d_out=x.data_ptr(),
            out_stride=self.DIM, out_dtype=pkg.DTYPE_BF16), self.stream())
        kv = (x @ self.wkv.t()).view(cap, 2 * self.KV, self.HEAD)
        slot = torch.empty(cap, dtype=torch.int64, device="cuda")
        tok.paged_assign_device(pkg.PagedArgs(
            d_item_off=off.data_ptr(), d_ctx_len=self.seq.data_ptr(), n=self.n, block_size=self.BLOCK, d_table=self.table.data_ptr(),
            table_stride=self.max_blocks, max_blocks=self.max_blocks, d_free=self.free.data_ptr(), d_n_free=self.n_free.data_ptr(),
            d_n_free_out=self.n_free.data_ptr(), d_slot=slot.data_ptr(), cap=cap, d_seq_len=self.seq.data_ptr(),
            d_status=self.status.data_ptr()), self.stream())
        tok.paged_store_device(self.cache(), pkg.StoreArgs(
            d_k=kv.data_ptr(), d_v=kv[:, self.KV:].data_ptr(), token_stride=kv.stride(0), head_stride=kv.stride(1),
            d_slot=slot.data_ptr(), n=cap), self.stream())
        self.keep += [x, kv, slot]
        return x

    def cache(self):
        return self.pkg.KVCache(d_k=self.k.data_ptr(), d_v=self.v.data_ptr(), block_stride=self.k.stride(0), token_stride=self.k.stride(1),
                                head_stride=self.k.stride(2), dtype=self.pkg.DTYPE_BF16, n_blocks=self.n_blocks,
                                block_size=self.BLOCK, kv_heads=self.KV, head_dim=self.HEAD)

    def step(self):
        """One token of each request, from self.ids to self.ids."""
        torch, pkg, tok, n = self.torch, self.pkg, self.tok, self.n
        self.x = self.rows(self.ids, self.one_off, n)
        self.q = (self.x @ self.wq.t()).view(n, self.HEADS, self.HEAD)
        tok.paged_attend_device(self.cache(), pkg.AttendArgs(
            d_q=self.q.data_ptr(), q_stride=self.q.stride(0), q_head_stride=self.HEAD, d_out=self.out.data_ptr(),
            out_stride=self.out.stride(0), out_head_stride=self.HEAD, n=n, heads=self.HEADS, scale=self.HEAD ** -0.5,
            d_table=self.table.data_ptr(), table_stride=self.max_blocks, max_blocks=self.max_blocks, d_seq_len=self.seq.data_ptr(),
            d_work=self.work.data_ptr(), work_bytes=self.work.numel()), self.stream())
        hidden = self.x + self.out.view(n, -1) @ self.wo.t()
        torch.mm(hidden, self.head.t(), out=self.logits)
        tok.process_logits_device(pkg.LogitsArgs(
            d_logits=self.logits.data_ptr(), logits_stride=self.V, d_out=self.scores.data_ptr(), out_stride=self.V,
            dtype=pkg.DTYPE_BF16, rows=n, n_logits=self.V, d_temperature=self.temperature.data_ptr()), self.stream())
        tok.sample_device(pkg.SampleArgs(
            d_scores=self.scores.data_ptr(), scores_stride=self.V, dtype=pkg.DTYPE_BF16, rows=n, n_logits=self.V,
            d_top_k=self.top_k.data_ptr(), d_top_p=self.top_p.data_ptr(), d_random=self.random.data_ptr(),
            d_pick=self.ids.data_ptr(), d_kept=self.kept.data_ptr(), d_logprob=self.logprob.data_ptr()), self.stream())
        self.keep += [self.x, self.q]


def test_decode(request):
    import torch

    from exact_bpe_tokenization_utf_gb300 import _build
    _build.build()
    import exact_bpe_tokenization_utf_gb300 as pkg
    from test_gpu_sample import _plain
    tok = pkg.Tokenizer.from_merges([], pkg.PATTERN_GPT2)
    request.addfinalizer(tok.close)
    rng = np.random.default_rng(0)
    prompts = [rng.integers(0, 1257, m).tolist() for m in (37, 1, 16, 200)]
    m = _Model(torch, pkg, tok, prompts)
    # the prompts but for their last tokens, which the first step takes
    for p in range(len(prompts)):
        m.ids[p] = prompts[p][-1]
    head = torch.tensor([t for p in prompts for t in p[:-1]], dtype=torch.int32, device="cuda")
    off = torch.tensor(np.concatenate([[0], np.cumsum([len(p) - 1 for p in prompts])]), device="cuda")
    m.rows(head, off, len(head))
    # a first step outside a graph, on copies, so that libraries are set up
    state = [t.clone() for t in (m.ids, m.seq, m.table, m.n_free, m.k, m.v)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for t, old in zip((m.ids, m.seq, m.table, m.n_free, m.k, m.v), state):
        t.copy_(old)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step()
    history = [list(p[:-1]) for p in prompts]
    for step in range(m.STEPS):
        ids = m.ids.tolist()
        m.random.copy_(torch.from_numpy(rng.random(len(prompts)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        for r, t in enumerate(ids):
            history[r].append(t)
        assert m.seq.tolist() == [len(h) for h in history]
        # rows
        want = m.embed[torch.tensor(ids, device="cuda").long()].double() * float(np.float32(m.DIM ** 0.5))
        assert bool(((m.x.double() - want).abs() <= want.abs() * 2.0**-8 * 1.01).all())
        # attention over the whole history, computed from the ids
        for r, h in enumerate(history):
            rows = (m.embed[torch.tensor(h, device="cuda")].float() * np.float32(m.DIM ** 0.5)).bfloat16()
            p = torch.arange(len(h), device="cuda")
            k, v = (t[m.table[r, p // m.BLOCK].long(), p % m.BLOCK] for t in (m.k, m.v))
            kv = (rows.double() @ m.wkv.double().t()).view(len(h), 2, m.KV, m.HEAD)
            size = (rows.double().abs() @ m.wkv.double().abs().t()).view(len(h), 2, m.KV, m.HEAD)
            for got, w, z in ((k, kv[:, 0], size[:, 0]), (v, kv[:, 1], size[:, 1])):   # (a library product, rounded to bf16)
                assert bool(((got.double() - w).abs() <= w.abs() * 2.0**-8 * 1.01 + z * m.DIM * 2.0**-23).all())
            q = m.q[r].double().view(m.KV, -1, m.HEAD)
            s = torch.einsum("hgd,thd->hgt", q, k.double()) * m.HEAD ** -0.5
            w = torch.softmax(s, 2)
            out = torch.einsum("hgt,thd->hgd", w, v.double()).reshape(m.HEADS, m.HEAD)
            room = torch.einsum("hgt,thd->hgd", w, v.double().abs()).reshape(m.HEADS, m.HEAD)
            off_by = max(1.0, float(s.abs().max()) * 40) * 2.0**-19
            assert bool(((m.out[r].double() - out).abs() <= out.abs() * 2.0**-8 * 1.01 + room * off_by).all())
        # the choice
        x = m.scores.float().cpu().numpy()
        for r in range(m.n):
            pick, kept, lp = _plain(x[r], top_k=int(m.top_k[r]), top_p=float(m.top_p[r]), u=float(m.random[r]))
            assert (int(m.ids[r]), int(m.kept[r])) == (pick, kept)
            assert abs(float(m.logprob[r]) - lp) <= 2.0**-24 * abs(lp) + 2.0**-30
    # the gradient of the embedding from all tokens of the run
    tokens = torch.tensor([t for h in history for t in h], dtype=torch.int32, device="cuda")
    grad = torch.randn(len(tokens), m.DIM, device="cuda").bfloat16()
    gw = torch.empty(m.V, m.DIM, device="cuda")
    work = torch.empty(tok.embed_work_bytes(len(tokens), m.V, m.DIM), dtype=torch.uint8, device="cuda")
    tok.embed_backward_device(pkg.EmbedGradArgs(
        d_ids=tokens.data_ptr(), n=len(tokens), n_rows=m.V, dim=m.DIM, scale=m.DIM ** 0.5, d_grad_out=grad.data_ptr(),
        grad_out_stride=m.DIM, grad_out_dtype=pkg.DTYPE_BF16, d_grad_weight=gw.data_ptr(), grad_weight_stride=m.DIM,
        grad_weight_dtype=pkg.DTYPE_F32, d_work=work.data_ptr(), work_bytes=work.numel()), m.stream())
    want = torch.zeros(m.V, m.DIM, dtype=torch.float64, device="cuda").index_add_(0, tokens.long(), grad.double()) * m.DIM ** 0.5
    size = torch.zeros(m.V, m.DIM, dtype=torch.float64, device="cuda").index_add_(0, tokens.long(), grad.double().abs()) * m.DIM ** 0.5
    assert bool(((gw.double() - want).abs() <= size * (len(tokens) + 3) * 2.0**-24).all())
