"""The serving calls on the host (no GPU needed): every refusal comes before any CUDA call, with its status and a
message; the Python layer checks layouts that the C ABI cannot see."""
import copy
import ctypes
import importlib.util
import math
import os
import pickle
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000   # aligned, never dereferenced


def _gpu():
    return torch.cuda.is_available()


def _plan(adt, rot=64, **kw):
    return adt.RopePlan(rot, **kw)


def test_plan_refusals(adt):
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=258), dict(rot_dim=64, base=1.0),
               dict(rot_dim=64, base=float("nan")), dict(rot_dim=64, base=float("inf")),
               dict(rot_dim=64, scaling="linear", factor=0.5), dict(rot_dim=64, scaling="ntk", factor=float("inf")),
               dict(rot_dim=64, scaling="yarn", factor=2.0, orig_len=0),
               dict(rot_dim=64, scaling="yarn", factor=2.0, orig_len=10, beta_fast=1.0, beta_slow=1.0),
               dict(rot_dim=64, scaling="yarn", factor=2.0, orig_len=10, beta_slow=0.0),
               dict(rot_dim=4, axis=[0, 8])):
        with pytest.raises(adt.SageError) as e:
            adt.RopePlan(**kw)
        assert e.value.status == 1 and len(str(e.value)) > 30
    for kw in (dict(scaling="other"), dict(axis=[0]), dict(inv_freq=[1.0])):
        with pytest.raises(ValueError):
            adt.RopePlan(64, **kw)
    assert adt._lib.sage_rope_plan_init(None, 64, 0, 10000.0, 0, 1.0, 0, 32.0, 1.0, None) == 1
    bad = adt.SageRopePlan()
    assert adt._lib.sage_rope_plan_init(ctypes.byref(bad), 64, 0, 10000.0, 9, 1.0, 0, 32.0, 1.0, None) == 1


def test_plan_formulas(adt):
    r, base, s, L0 = 96, 10000.0, 8.0, 4096
    want = [base ** (-2 * i / r) for i in range(r // 2)]
    turns = lambda p: [t * 2 * math.pi for t in p.struct.turns[: r // 2]]  # noqa: E731
    assert turns(_plan(adt, r)) == pytest.approx(want, rel=1e-14)
    assert turns(_plan(adt, r, scaling="linear", factor=s)) == pytest.approx([f / s for f in want], rel=1e-14)
    b2 = base * s ** (r / (r - 2))
    assert turns(_plan(adt, r, scaling="ntk", factor=s)) == pytest.approx([b2 ** (-2 * i / r) for i in range(r // 2)],
                                                                           rel=1e-13)
    p = _plan(adt, r, scaling="yarn", factor=s, orig_len=L0, beta_fast=20, beta_slow=2)
    ramp = [min(1, max(0, (L0 * f / (2 * math.pi) - 2) / 18)) for f in want]
    assert turns(p) == pytest.approx([g * f + (1 - g) * f / s for g, f in zip(ramp, want)], rel=1e-13)
    assert 0 in ramp and 1 in ramp and any(0 < g < 1 for g in ramp)
    assert p.struct.mscale == pytest.approx(0.1 * math.log(s) + 1, rel=1e-6)
    # the last pair of an NTK plan turns `factor` times slower, the first as before
    ntk = turns(_plan(adt, r, scaling="ntk", factor=s))
    assert ntk[0] == pytest.approx(want[0]) and ntk[-1] == pytest.approx(want[-1] / s, rel=1e-12)
    assert _plan(adt, 2, scaling="ntk", factor=s).struct.turns[0] * 2 * math.pi == pytest.approx(1.0)
    axes = _plan(adt, 8, axis=[0, 2, 1, 2])
    assert axes.n_axes == 3 and list(axes.struct.axis[:4]) == [0, 2, 1, 2]
    assert _plan(adt, 8, mscale=0.5).struct.mscale == 0.5


def test_rope_refusals(adt):
    L = adt._lib
    plan = _plan(adt, 64)

    def call(q=(FAKE, FAKE, 4, 0, 0), k=(FAKE, FAKE, 2, 0, 0), T=3, D=64, dt=0, pos=FAKE, pl=plan.struct):
        return L.sage_rope(adt.SageRows(*q), adt.SageRows(*k), T, D, dt, pos, None if pl is None else ctypes.byref(pl),
                           0, None)

    assert call(pl=None) == 1
    assert call(T=-1) == 1
    assert call(D=60) == 2 and call(D=264) == 2 and call(D=0) == 2
    assert call(dt=3) == 1
    assert call(D=56) == 1                                    # rot_dim above D
    assert call(q=(FAKE, FAKE, -1, 0, 0)) == 1
    assert call(q=(None, FAKE, 4, 0, 0)) == 1 and call(k=(FAKE, None, 2, 0, 0)) == 1
    assert call(q=(FAKE + 8, FAKE, 4, 0, 0)) == 3
    assert call(q=(FAKE, FAKE, 4, 255, 0)) == 1 and call(q=(FAKE, FAKE, 4, 260, 0)) == 3
    assert call(q=(FAKE, FAKE, 4, 512, 256)) == 1             # in place with two strides
    assert call(pos=None) == 1 and call(pos=FAKE + 4) == 3
    for field, value in (("rot_dim", 63), ("n_axes", 0), ("n_axes", 9)):
        bad = adt.SageRopePlan.from_buffer_copy(plan.struct)
        setattr(bad, field, value)
        assert call(pl=bad) == 1, field
    bad = adt.SageRopePlan.from_buffer_copy(plan.struct)
    bad.axis[5] = 1
    assert call(pl=bad) == 1 and b"axis" in L.sage_last_error()
    bad = adt.SageRopePlan.from_buffer_copy(plan.struct)
    bad.turns[0] = float("nan")
    assert call(pl=bad) == 1
    assert call(T=0, q=(None, None, 4, 0, 0), k=(None, None, 2, 0, 0), pos=None) == 0
    assert call(q=(None, None, 0, 0, 0), k=(None, None, 0, 0, 0)) == 0
    if not _gpu():
        assert call() == 4


def _cache(adt, **over):
    a = dict(k_codes=FAKE, k_scale=FAKE, v_codes=FAKE, v_scale=FAKE, num_pages=4, page_size=16, Hk=2, D=64, format=0)
    a.update(over)
    return adt.SageKvCache(*[a[f] for f, _ in adt.SageKvCache._fields_])


BAD_CACHES = [(dict(num_pages=0), 1), (dict(Hk=0), 1), (dict(page_size=8), 2), (dict(page_size=24), 2),
              (dict(page_size=2048), 2), (dict(D=96), 2), (dict(format=2), 1), (dict(k_codes=None), 1),
              (dict(v_scale=None), 1), (dict(v_codes=FAKE + 8), 3), (dict(k_scale=FAKE + 4), 3)]


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_cache_refusals(adt, over, status):
    L, c = adt._lib, _cache(adt, **over)
    assert L.sage_kv_write(FAKE, FAKE, 3, 0, 0, 0, FAKE, c, None) == status
    assert L.sage_kv_read(c, FAKE, 3, FAKE, FAKE, 0, 0, 0, None) == status
    p = adt.SageToken(1, 4, 0, 0, 0, FAKE, 4, FAKE, 64, 0.0)
    assert L.sage_attn_token(FAKE, ctypes.byref(p), c, FAKE, None, FAKE << 8, 1 << 30, None) == status


def test_write_and_read_refusals(adt):
    L, c = adt._lib, _cache(adt)

    def both(status, k=FAKE, v=FAKE, T=3, ks=0, vs=0, dt=0, slots=FAKE, c=c):
        assert L.sage_kv_write(k, v, T, ks, vs, dt, slots, c, None) == status
        assert L.sage_kv_read(c, slots, T, k, v, ks, vs, dt, None) == status

    both(1, T=-1)
    both(1, dt=7)
    both(1, k=None)
    both(3, v=FAKE + 2)
    both(1, slots=None)
    both(3, slots=FAKE + 4)
    both(1, ks=64)
    both(3, vs=129)
    both(1, T=(1 << 31) - 1)
    both(0, T=0, k=None, v=None, slots=None)
    if not _gpu():
        both(4)


def _prompt(adt, cu_q, cu_k=None, **over):
    a = dict(Hq=4, Hk=2, D=64, q_stride=0, k_stride=0, v_stride=0, out_stride=0, dtype=0, causal=1, sm_scale=0.0)
    a.update(over)
    arrs = [None if c is None else (ctypes.c_int32 * len(c))(*c) for c in (cu_q, cu_k)]
    p = adt.SagePrompt(a.pop("n_seq", len(cu_q) - 1 if cu_q else 1), *[None if x is None else ctypes.addressof(x) for x in arrs],
                       a["Hq"], a["Hk"], a["D"], a["q_stride"], a["k_stride"], a["v_stride"], a["out_stride"],
                       a["dtype"], a["causal"], a["sm_scale"])
    p._keep = arrs
    return p


def test_prompt_refusals(adt):
    L = adt._lib

    def call(p, q=FAKE, k=FAKE, v=FAKE, out=2 * FAKE, lse=None):
        return L.sage_attn_prompt(q, k, v, None if p is None else ctypes.byref(p), out, lse, None)

    ok = [0, 3, 10]
    assert call(None) == 1
    assert call(_prompt(adt, ok, n_seq=-1)) == 1
    assert call(_prompt(adt, None)) == 1
    for cu in ([1, 3], [0, 5, 3]):
        assert call(_prompt(adt, cu)) == 1 and call(_prompt(adt, [0] * len(cu), cu)) == 1
    assert call(_prompt(adt, ok, Hq=3)) == 1 and call(_prompt(adt, ok, Hk=0)) == 1 and call(_prompt(adt, ok, Hq=0)) == 1
    assert call(_prompt(adt, ok, D=96)) == 2
    assert call(_prompt(adt, ok, dtype=2)) == 2
    for s in (float("nan"), float("inf"), float("-inf")):
        assert call(_prompt(adt, ok, sm_scale=s)) == 1
    for name in ("q_stride", "out_stride"):
        assert call(_prompt(adt, ok, **{name: 128})) == 1 and call(_prompt(adt, ok, **{name: 260})) == 3
    for name in ("k_stride", "v_stride"):
        assert call(_prompt(adt, ok, **{name: 64})) == 1 and call(_prompt(adt, ok, **{name: 132})) == 3
    for name in ("q", "k", "v", "out"):
        assert call(_prompt(adt, ok), **{name: None}) == 1 and call(_prompt(adt, ok), **{name: FAKE + 2}) == 3
    assert call(_prompt(adt, ok), lse=FAKE + 2) == 3
    for name in ("q", "k", "v"):                                   # out on top of an input
        ptrs = dict(q=FAKE, k=2 * FAKE, v=3 * FAKE, out=4 * FAKE)
        ptrs["out"] = ptrs[name]
        assert call(_prompt(adt, ok), **ptrs) == 1 and b"out" in L.sage_last_error()
    assert call(_prompt(adt, [0]), q=None) == 0 and call(_prompt(adt, [0, 0], [0, 7]), q=None) == 0
    if not _gpu():
        assert call(_prompt(adt, ok)) == 4
        assert call(_prompt(adt, ok, [0, 0, 0]), k=None, v=None) == 4      # no keys: K and V are not needed


def test_token_refusals(adt):
    L, c = adt._lib, _cache(adt)

    def call(q=FAKE, out=FAKE, lse=None, ws=FAKE << 8, wsb=1 << 30, c=c, null=False, **over):
        a = dict(B=2, Hq=4, q_stride=0, out_stride=0, dtype=0, page_table=FAKE, table_stride=40, lens=FAKE, max_len=640,
                 sm_scale=0.0)
        a.update(over)
        p = adt.SageToken(*[a[f] for f, _ in adt.SageToken._fields_])
        return L.sage_attn_token(q, None if null else ctypes.byref(p), c, out, lse, ws, wsb, None)

    assert call(null=True) == 1
    assert call(Hq=3) == 1 and call(Hq=0) == 1
    assert call(B=-1) == 1 and call(B=70000) == 1
    assert call(dtype=2) == 2
    assert call(sm_scale=float("nan")) == 1
    assert call(q_stride=128) == 1 and call(out_stride=257) == 3
    assert call(max_len=641) == 1 and call(max_len=-1) == 1 and call(table_stride=-1) == 1
    assert call(q=None) == 1 and call(out=FAKE + 8) == 3
    assert call(lens=None) == 1 and call(page_table=None) == 1
    assert call(lens=FAKE + 2) == 3 and call(page_table=FAKE + 1) == 3 and call(lse=FAKE + 2) == 3
    need = adt.attn_token_workspace_bytes(2, 4, 2, 64, 640)
    assert need > 0 and need % 256 == 0
    assert call(ws=None) == 6 and call(ws=(FAKE << 8) + 16) == 3 and call(wsb=need - 1) == 6
    assert call(B=0, q=None, lens=None, page_table=None, ws=None) == 0
    assert call(c=_cache(adt, Hk=40000), Hq=40000 * 17) == 1                # too many heads
    if not _gpu():
        assert call(wsb=need) == 4
        assert call(max_len=0, page_table=None, ws=None) == 4               # no keys at all
    assert adt.attn_token_workspace_bytes(2, 3, 2, 64, 640) == 0            # Hq no multiple of Hk
    assert adt.attn_token_workspace_bytes(2, 4, 2, 96, 640) == 0
    assert adt.attn_token_workspace_bytes(0, 4, 2, 64, 640) == 0


def test_python_layer_refuses_layouts(adt):
    """Layouts are checked before the device: these tensors are on the CPU, and each call names its fault."""
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    plan = adt.RopePlan(64)
    cache = adt.KVCache(2, 16, 2, 64, device="cpu")
    kc, ks, vc, vs = cache.tensors
    table, lens = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="fmt"):
        adt.KVCache(2, 16, 2, 64, fmt="int4", device="cpu")

    def rope(q=x, k=x, pos=slots, **kw):
        adt.sage_rope(q, k, pos, plan, **kw)

    def write(k=x, v=x, sl=slots, c=(kc, ks, vc, vs)):
        adt.sage_kv_write(k, v, sl, *c)

    def read(k=x, v=x, sl=slots, c=(kc, ks, vc, vs)):
        adt.sage_kv_read(sl, *c, k, v)

    def prompt(q=x, k=x, v=x, cu=(0, 3), **kw):
        adt.sage_attn_prompt(q, k, v, cu, **kw)

    def token(q=x, c=(kc, ks, vc, vs), t=table, ln=lens, out=x, ws=None, **kw):
        adt.sage_attn_token(q, *c, t, ln, out, ws, **kw)

    for call in (rope, write, read, prompt, token):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    wide, narrow = torch.zeros(3, 64, 2, dtype=torch.bfloat16).transpose(1, 2), torch.zeros(3, 2, 32, dtype=torch.bfloat16)
    for bad, kind, word in ((wide, ValueError, "strides"), (narrow, ValueError, "must be"), (x[0], ValueError, "must be"),
                            (x[:1].expand(3, 2, 64), ValueError, "stride 0"), (x.double(), TypeError, "dtype|beside|Double"),
                            (7, TypeError, "tensor")):
        for call in (rope, write, read, prompt):
            with pytest.raises(kind, match=word if not (call is rope and bad is narrow) else "must be"):
                call(k=bad)
    for call in (write, read, prompt):
        with pytest.raises(TypeError, match="beside"):
            call(v=x.half())
    with pytest.raises(ValueError, match="q or k"):
        rope(q=None, k=None)
    with pytest.raises(ValueError, match="q_out"):
        rope(q_out=narrow)
    with pytest.raises(TypeError, match="tensor"):
        rope(q=None, q_out=5)
    with pytest.raises(ValueError, match="positions"):
        rope(pos=slots.int())
    with pytest.raises(ValueError, match="positions"):
        rope(pos=slots[:2])
    with pytest.raises(ValueError, match="positions"):
        rope(pos=torch.zeros(2, 3, dtype=torch.int64))
    for call in (write, read):
        for bad in (torch.zeros(6, dtype=torch.int64)[::2], slots.int(), slots[:2]):
            with pytest.raises(ValueError, match="slots"):
                call(sl=bad)
    for call in (write, read, token):
        for bad in ((kc.float(), ks, vc, vs), (kc, ks, vc.view(torch.uint8), vs), (kc, ks.double(), vc, vs)):
            with pytest.raises(TypeError):
                call(c=bad)
        for bad in ((kc, ks[:1], vc, vs), (kc.transpose(0, 1), ks, vc, vs), (kc[0], ks, vc[0], vs)):
            with pytest.raises(ValueError):
                call(c=bad)
    with pytest.raises(ValueError, match="contiguous"):
        write(c=(torch.zeros(2, 2, 32, 64, dtype=torch.int8)[:, :, ::2], ks, vc, vs))
    for bad in ((0, 2), [], [0, 1, 2], torch.tensor([0, 2])):
        with pytest.raises(ValueError, match="cu_q"):
            prompt(cu=bad)
    with pytest.raises(ValueError, match="cu_q"):
        prompt(cu=[0, -1, 3])
    with pytest.raises(ValueError, match="sequences"):
        prompt(cu_k=[0, 1, 3])
    with pytest.raises(TypeError):
        prompt(cu=5)
    for bad in (torch.zeros(3, 2), torch.zeros(2, 3, dtype=torch.float64), torch.zeros(3, 2).t()):
        with pytest.raises(ValueError, match="lse"):
            prompt(lse=bad)
    with pytest.raises(ValueError, match="out"):
        prompt(out=narrow)
    for bad in (table.long(), table[:2], table.t(), table[:1].expand(3, 2)):
        with pytest.raises(ValueError, match="page_table"):
            token(t=bad)
    with pytest.raises(ValueError, match="lens"):
        token(ln=lens.long())
    for bad in (33, -1):
        with pytest.raises(ValueError, match="max_len"):
            token(max_len=bad)
    with pytest.raises(ValueError, match="lse"):
        token(lse=torch.zeros(2, 3))
    with pytest.raises(ValueError, match="workspace"):
        token(ws=torch.zeros(64)[::2])
    with pytest.raises(ValueError, match="q must be|out must be"):
        token(q=narrow)


@pytest.mark.parametrize("Hq,Hk,D", [(32, 8, 128), (4, 4, 64), (40, 1, 64), (512, 8, 128), (1, 1, 128)])
def test_a_workspace_serves_fewer_and_shorter_sequences(adt, Hq, Hk, D):
    """A batch that thins out, or a tighter max_len, needs no more than the largest one asked for; the call itself takes
    what its own chunks need (checked on the host, in front of the launch)."""
    need = lambda B, L: adt.attn_token_workspace_bytes(B, Hq, Hk, D, L)  # noqa: E731
    lens = [0, 1, 32, 128, 129, 384, 512, 1000, 2047, 2048, 2049, 8192, 100000]
    batches = [1, 2, 3, 8, 16, 27, 32, 55, 56, 64, 111, 222, 443, 444, 445, 1000]
    for i, B in enumerate(batches):
        for j, L in enumerate(lens):
            assert need(B, L) >= max([need(b, L) for b in batches[:i]] + [need(B, x) for x in lens[:j]] + [0]), (B, L)
    if _gpu():
        return                                                   # valid calls on made-up addresses: only without a GPU
    c = _cache(adt, Hk=Hk, D=D, num_pages=1 << 20, page_size=64)
    for B, L in ((64, 2048), (27, 8192), (444, 100000), (1000, 512)):
        ws = need(B, L)
        for b in batches:
            for x in lens:
                if b <= B and x <= L:
                    p = adt.SageToken(b, Hq, 0, 0, 0, FAKE, 4096, FAKE, x, 0.0)
                    st = adt._lib.sage_attn_token(FAKE, ctypes.byref(p), c, FAKE, None, FAKE << 8 if ws else None, ws, None)
                    assert st == 4, (B, L, b, x)


def test_the_library_serves_without_the_extension_module(adt):
    """The quantized attention needs libsage.so alone; a serving call names what is missing and how to build it."""
    code = """if True:
        import sys
        sys.modules["action_diffusion_transformers_b200._serve_ext"] = None        # fails to import
        import torch, action_diffusion_transformers_b200 as adt
        assert adt.npad(130) == 256 and adt.RopePlan(64).rot_dim == 64
        x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
        c = adt.KVCache(1, 16, 2, 64, device="cpu")
        for call in (lambda: adt.sage_attn_prompt(x, x, x, [0, 1]), lambda: c.write(x, x, torch.zeros(1).long()),
                     lambda: adt.sage_rope(x, x, torch.zeros(1).long(), adt.RopePlan(64))):
            try:
                call()
                assert False
            except ImportError as e:
                assert "_serve_ext" in str(e) and "build" in str(e)
        print("fine")
    """
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_the_extension_module_is_built_again_for_another_torch(adt, monkeypatch):
    spec = importlib.util.spec_from_file_location("_build_of_the_module", os.path.join(os.path.dirname(adt.LIB_PATH), "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    assert b.up_to_date()
    assert torch.__version__ in b.built_for() and adt._serve_ext.__doc__.endswith(b.built_for())
    for other in (b.built_for() + ".1", b.built_for().replace("torch 2", "torch 3"), "torch 1.0"):
        monkeypatch.setattr(b, "built_for", lambda other=other: other)
        assert not b.up_to_date()


def test_a_copied_plan_is_its_own(adt):
    """Plans travel with the modules that hold them: a copy names its own struct, not the first one's (which may be gone)."""
    first = _plan(adt, 64, scaling="yarn", factor=4.0, orig_len=256)
    for again in (copy.deepcopy(first), pickle.loads(pickle.dumps(first))):
        assert again.address == ctypes.addressof(again.struct) != first.address
        assert bytes(again.struct) == bytes(first.struct)
        again.struct.mscale = 2.0
        assert first.struct.mscale != 2.0


def test_token_attention_in_place_needs_one_stride(adt):
    c = _cache(adt)
    for qs, os_, status in ((256, 512, 1), (0, 512, 1), (512, 256, 1)):
        p = adt.SageToken(2, 4, qs, os_, 0, FAKE, 40, FAKE, 640, 0.0)
        assert adt._lib.sage_attn_token(FAKE, ctypes.byref(p), c, FAKE, None, FAKE << 8, 1 << 30, None) == status
        assert b"stride" in adt._lib.sage_last_error()
