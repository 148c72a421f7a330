"""The serving operators together, as a conditioner uses them: rotate, write to the cache, attend over the prompt; read
the context back for the next part of the prompt; then go on token by token.  Plus guard bytes around every output."""
import pytest
import torch

from tests.serve_ref import attend, check
from tests.test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu


class Layer:
    """Attention state of a batch: one cache, one page table; K is rotated before it is cached."""

    def __init__(self, adt, B, Hq, Hk, D, ps, fmt, dtype, longest):
        self.adt, self.B, self.Hq, self.Hk, self.D, self.ps, self.dtype = adt, B, Hq, Hk, D, ps, dtype
        per = -(-longest // ps)
        self.cache = adt.KVCache(B * per, ps, Hk, D, fmt)
        self.table = torch.randperm(B * per, generator=torch.Generator().manual_seed(1)).int().view(B, per).cuda()
        self.plan = adt.RopePlan(D, scaling="yarn", factor=4.0, orig_len=256)
        self.lens = [0] * B
        self.ws = torch.empty(max(256, adt.attn_token_workspace_bytes(B, Hq, Hk, D, per * ps)), dtype=torch.uint8,
                              device="cuda")

    def places(self, counts):
        """Positions and slots of the next counts[b] tokens of each sequence."""
        pos = torch.cat([torch.arange(n, n + c) for n, c in zip(self.lens, counts)]).cuda()
        seq = torch.cat([torch.full((c,), b) for b, c in enumerate(counts)]).cuda()
        return pos, self.table.long()[seq, pos // self.ps] * self.ps + pos % self.ps

    def context(self):
        """The cached context of every sequence, packed."""
        seq = torch.cat([torch.full((n,), b) for b, n in enumerate(self.lens)]).cuda()
        pos = torch.cat([torch.arange(n) for n in self.lens]).cuda()
        slots = self.table.long()[seq, pos // self.ps] * self.ps + pos % self.ps
        k = torch.empty(len(slots), self.Hk, self.D, dtype=self.dtype, device="cuda")
        return self.cache.read(slots, k, torch.empty_like(k))

    def part(self, q, k, v, counts):
        """counts[b] more tokens of each prompt: rotate, write, attend to the context as the cache holds it."""
        pos, slots = self.places(counts)
        self.adt.sage_rope(q, k, pos, self.plan)
        self.cache.write(k, v, slots)
        self.lens = [n + c for n, c in zip(self.lens, counts)]
        kc, vc = self.context()
        cu = lambda ns: [sum(ns[:i]) for i in range(len(ns) + 1)]  # noqa: E731
        return self.adt.sage_attn_prompt(q, kc, vc, cu(counts), cu(self.lens)), kc, vc

    def token(self, q, k, v, out, lse):
        pos, slots = self.places([1] * self.B)
        self.adt.sage_rope(q, k, pos, self.plan)
        self.cache.write(k, v, slots)
        self.lens = [n + 1 for n in self.lens]
        lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        return self.cache.attend(q, self.table, lens, out, self.ws, lse=lse)


@pytest.mark.parametrize("fmt,dtype,D", [("int8", torch.bfloat16, 128), ("e4m3", torch.float16, 64)])
def test_prompt_in_parts_then_tokens(adt, fmt, dtype, D):
    B, Hq, Hk, ps = 3, 8, 2, 32
    lay = Layer(adt, B, Hq, Hk, D, ps, fmt, dtype, 512)
    g = torch.Generator(device="cuda").manual_seed(2)

    def rows(n):
        qkv = torch.randn(n, (Hq + 2 * Hk) * D, generator=g, device="cuda").to(dtype)
        return (qkv[:, : Hq * D].view(n, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(n, Hk, D),
                qkv[:, (Hq + Hk) * D:].view(n, Hk, D))

    half = torch.finfo(dtype).eps / 2
    for counts in ([150, 7, 64], [33, 200, 1]):
        q, k, v = rows(sum(counts))
        out, kc, vc = lay.part(q, k, v, counts)
        a = c = 0
        for b, n in enumerate(counts):
            L = lay.lens[b]
            vis = torch.arange(n, device="cuda") + 1 + L - n
            for h in range(Hq):
                ref = attend(q[a:a + n, h].double(), kc[c:c + L, h // 4].double(), vc[c:c + L, h // 4].double(), vis,
                             D ** -0.5, half)
                check(out[a:a + n, h], None, *ref, what=(b, h))
            a, c = a + n, c + L
    # single tokens: the cache attention equals the prompt attention of one query over the context read back, to the
    # two kernels' own roundings (P in 16 bits in each; the context rounded to 16 bits by the read)
    out, lse = torch.empty(B, Hq, D, dtype=dtype, device="cuda"), torch.empty(B, Hq, device="cuda")
    for _ in range(4):
        q, k, v = rows(B)
        lay.token(q, k, v, out, lse)
        kc, vc = lay.context()
        cu = [sum(lay.lens[:i]) for i in range(B + 1)]
        lse2 = torch.empty(Hq, B, device="cuda")
        out2 = adt.sage_attn_prompt(q, kc, vc, list(range(B + 1)), cu, lse=lse2)
        for b in range(B):
            for h in range(Hq):
                x, y = kc[cu[b]:cu[b + 1], h // 4].double(), vc[cu[b]:cu[b + 1], h // 4].double()
                o, l, tol, tl = attend(q[b, h][None].double(), x, y, torch.tensor([lay.lens[b]], device="cuda"),
                                       D ** -0.5, half)
                check(out2[b, h][None], lse2[h, b][None], o, l, tol, tl)
                # reading rounds K and V by half a step: the score moves by half * scale * |q| . |k|, V by half of itself
                s = half * D ** -0.5 * float((q[b, h].double().abs() @ x.abs().t()).max())
                A = tol / (half + 2.0 ** -19)
                check(out[b, h][None], lse[b, h][None], o, l, tol + A * (2.0 ** -11 + half + 2 * s), tl + s)
    adt.sage_check()


def test_decode_step_as_one_graph(adt):
    """Rotate, write and attend of one decoding step captured once and replayed for every token, the positions, slots
    and lengths changing in place: the same bits as eager calls."""
    B, Hq, Hk, D, ps = 2, 8, 2, 64, 16
    results = []
    for use_graph in (False, True):
        lay = Layer(adt, B, Hq, Hk, D, ps, "int8", torch.bfloat16, 128)
        g = torch.Generator(device="cuda").manual_seed(5)
        qkv = torch.empty(B, (Hq + 2 * Hk) * D, dtype=torch.bfloat16, device="cuda")
        q, k, v = (qkv[:, : Hq * D].view(B, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(B, Hk, D),
                   qkv[:, (Hq + Hk) * D:].view(B, Hk, D))
        pos, slots = torch.zeros(B, dtype=torch.int64, device="cuda"), torch.full((B,), -1, device="cuda")
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        qr, kr = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B, Hk, D, dtype=torch.bfloat16, device="cuda")
        out = torch.empty_like(qr)

        def step():
            adt.sage_rope(q, k, pos, lay.plan, qr, kr)
            lay.cache.write(kr, v, slots)
            lay.cache.attend(qr, lay.table, lens, out, lay.ws)

        step()                                                   # every one-time setup outside the capture
        if use_graph:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        outs = []
        for t in range(40):
            qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
            p, sl = lay.places([1] * B)
            lay.lens = [n + 1 for n in lay.lens]
            pos.copy_(p)
            slots.copy_(sl)
            lens.copy_(torch.tensor(lay.lens, dtype=torch.int32))
            graph.replay() if use_graph else step()
            outs.append(out.clone())
        adt.sage_check()
        results.append(torch.stack(outs))
    assert torch.equal(results[0], results[1])


@pytest.mark.parametrize("D,dtype", [(64, torch.bfloat16), (128, torch.float16)])
def test_no_write_outside_the_buffers(adt, D, dtype):
    Hq, Hk, ps, T = 6, 2, 16, 131
    x = torch.randn(T, Hq, D, device="cuda").to(dtype)
    y = torch.randn(T, Hk, D, device="cuda").to(dtype)
    pos = torch.arange(T, device="cuda")
    gs = []

    def new(shape, dt):
        gs.append(Guarded(shape, dt))
        return gs[-1].t

    for rot, pairs in ((D, True), (D, False), (40, False), (14, False), (6, True)):
        adt.sage_rope(x, y, pos, adt.RopePlan(rot, interleaved=pairs), new((T, Hq, D), dtype), new((T, Hk, D), dtype))
    pages = 9
    kc, vc = new((pages, Hk, ps, D), torch.int8), new((pages, Hk, ps, D), torch.int8)
    ks, vs = new((pages, Hk, ps), torch.float32), new((pages, Hk, ps), torch.float32)
    slots = torch.arange(T, device="cuda") + 1
    adt.sage_kv_write(y, y, slots, kc, ks, vc, vs)
    adt.sage_kv_read(slots, kc, ks, vc, vs, new((T, Hk, D), dtype), new((T, Hk, D), dtype))
    adt.sage_attn_prompt(x, y, y, [0, 1, T], out=new((T, Hq, D), dtype), lse=new((Hq, T), torch.float32))
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(T, 1)
    lens = (torch.arange(T, device="cuda") % (pages * ps) + 0).int()
    ws = new((adt.attn_token_workspace_bytes(T, Hq, Hk, D, pages * ps) + 256,), torch.uint8)
    adt.sage_attn_token(x, kc, ks, vc, vs, table, lens, new((T, Hq, D), dtype), ws, lse=new((T, Hq), torch.float32))
    long = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(1, 40)
    ws = new((adt.attn_token_workspace_bytes(1, Hq, Hk, D, 360 * ps),), torch.uint8)
    adt.sage_attn_token(x[:1], kc, ks, vc, vs, long, torch.tensor([360 * ps - 3], dtype=torch.int32, device="cuda"),
                        new((1, Hq, D), dtype), ws)
    adt.sage_check()
    assert all(g.intact() for g in gs)
