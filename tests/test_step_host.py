"""Host-side checks of the operators around the layer (no GPU work): packed
structs match the header, bad arguments return an error and launch nothing."""
import ctypes
import os
import re
import subprocess
import sys
import types

import pytest
import torch

import top_routed_grouped_gb300 as moe
from top_routed_grouped_gb300 import build, step

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 256  # never read: the calls fail, or have no rows


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


def fields(name):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe.h")).read(), flags=re.S)
    body = re.search(r"typedef struct %s \{(.*?)\} %s_t;" % (name, name), src, flags=re.S).group(1)
    out = []
    for line in body.split(";"):
        line = line.strip()
        if line:
            kind, names = re.match(r"((?:const )?\w+ ?)\s*(.*)", line, flags=re.S).groups()
            for n in names.split(","):
                out.append((n.strip().lstrip("*"), "Q" if "*" in n else {"int32_t": "i", "float": "f", "int64_t": "q"}[kind.strip()]))
    return out


@pytest.mark.parametrize("name,packed", [("moe_norm_args", step._NORM), ("moe_embed_args", step._EMBED),
                                         ("moe_distill_args", step._DISTILL)])
def test_structs_match_the_header(name, packed):
    f = fields(name)
    letters = re.sub(r"(\d+)(\w)", lambda m: int(m.group(1)) * m.group(2), packed.format)
    assert "".join(k for _, k in f) == letters
    cls = type("S", (ctypes.Structure,), {"_fields_": [
        (n, {"i": ctypes.c_int32, "f": ctypes.c_float, "q": ctypes.c_int64, "Q": ctypes.c_void_p}[k]) for n, k in f]})
    assert ctypes.sizeof(cls) == packed.size


def packed(name, spec, **kw):
    base = {n: (PTR if k == "Q" else 0) for n, k in fields(name)}
    base.update(kw)
    return spec.pack(*[base[n] for n, _ in fields(name)])


def norm(**kw):
    return packed("moe_norm_args", step._NORM, **dict(dict(T=4, H=64, dtype=1, rdtype=1, wdtype=1, scale=1.0, eps=1e-6), **kw))


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), -1), (dict(H=0), -1), (dict(H=16385), -2), (dict(dtype=2), -1), (dict(rdtype=5), -1),
    (dict(dtype=0, rdtype=1), -1), (dict(dtype=0, rdtype=0, wdtype=1), -1), (dict(gate_kind=4), -1),
    (dict(scale=float("nan")), -1), (dict(eps=-1.0), -1), (dict(eps=float("inf")), -1), (dict(reserved=1), -1),
    (dict(ld_r=63), -1), (dict(ld_y=-64), -1), (dict(r=0), -1), (dict(r=PTR + 1), -1), (dict(h=0), -1),
    (dict(r_out=0), -1), (dict(y=0), -1), (dict(y=0, w_post=0, w_pre=0), -1), (dict(gate_kind=1, gate=0), -1),
    (dict(w_pre=PTR + 1), -1), (dict(T=0), 0), (dict(T=0, r=0, y=0, h=0), 0),
])
def test_norm_refusals(L, kw, want):
    assert L.moe_block_norm(norm(**kw), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dr=0), -1), (dict(dy=0), -1), (dict(dw_post=0), -1), (dict(dw_pre=0), -1), (dict(dh=0), -1),
    (dict(r_out=0), -1), (dict(dr_out=0, w_pre=0), -1), (dict(gate_kind=3, dgate=0), -1), (dict(H=1 << 20), -2),
])
def test_norm_backward_refusals(L, kw, want):
    assert L.moe_block_norm_backward(norm(**kw), PTR, 1 << 40, None) == want


@pytest.mark.parametrize("T,H", [(1, 1), (4, 64), (1000, 77), (5000, 256), (9, 4104), (70000, 2048), (33, 16384)])
def test_norm_workspace_goes_by_sizes(L, T, H):
    """One size, whether the buffers are there or not (run in a process of its
    own: a query that divides by zero takes the process with it), enough for
    any launch with the strides that it is asked for."""
    code = """if 1:
        import sys
        sys.path[:0] = [%r, %r]
        import top_routed_grouped_gb300 as moe, test_step_host as t
        L, n = moe.lib(), lambda **kw: moe.lib().moe_block_norm_workspace_size(t.norm(T=%d, H=%d, **kw))
        none = {k: 0 for k, kind in t.fields("moe_norm_args") if kind == "Q"}
        full = n()
        assert full %% 256 == 0  # (0 where there is no device)
        for kw in (none, dict(none, w_pre=t.PTR), dict(none, y=t.PTR), dict(y=0, w_post=0), dict(w_pre=0), dict(dr_out=0),
                   dict(y=t.PTR + 2), dict(gate_kind=3), dict(none, gate_kind=1), dict(dtype=0, rdtype=0, wdtype=0)):
            assert n(**kw) == full, kw
        assert n(ld_dh=%d) >= full
        assert L.moe_block_norm_workspace_size(t.norm(T=0)) == 0 and n(eps=-1.0) == 0
    """ % (ROOT, os.path.dirname(os.path.abspath(__file__)), T, H, H + 1)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])


def test_missing_arguments(L):
    assert L.moe_block_norm(None, None) == -1 and L.moe_block_norm_backward(None, None, 0, None) == -1
    assert L.moe_embed(None, None) == -1 and L.moe_embed_backward(None, None, 0, None) == -1
    assert L.moe_distill(None, None) == -1 and L.moe_block_norm_workspace_size(None) == 0
    assert L.moe_embed_workspace_size(None) == 0


def embed(**kw):
    return packed("moe_embed_args", step._EMBED, **dict(dict(T=4, H=64, V=100, dtype=1, odtype=1, scale=1.0, padding_id=-1), **kw))


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), -1), (dict(H=0), -1), (dict(V=0), -1), (dict(V=1 << 20), -2), (dict(dtype=3), -1),
    (dict(dtype=0, odtype=1), -1), (dict(ids=0), -1), (dict(ids=PTR + 2), -1), (dict(ids64=1, ids=PTR + 4), -1),
    (dict(ids64=2), -1), (dict(scale=float("inf")), -1), (dict(table=0), -1), (dict(out=PTR + 1), -1),
    (dict(ld_table=10), -1), (dict(T=0, ids=0, table=0, out=0), 0),
])
def test_embed_refusals(L, kw, want):
    assert L.moe_embed(embed(**kw), None) == want


def test_embed_backward_refusals(L):
    n = L.moe_embed_workspace_size(embed())
    assert n > 0 and n % 256 == 0
    for kw, ws, size, want in ((dict(dtable=0), PTR, n, -1), (dict(dout=0), PTR, n, -1), (dict(accumulate=2), PTR, n, -1),
                               ({}, PTR, n - 1, -3), ({}, 0, n, -1), ({}, PTR + 16, n, -1)):
        assert L.moe_embed_backward(embed(**kw), ws, size, None) == want


def distill(**kw):
    return packed("moe_distill_args", step._DISTILL, **dict(dict(T=4, V=100, K=3, dtype=1, temperature=1.0, scale=1.0), **kw))


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), -1), (dict(V=0), -1), (dict(K=0), -1), (dict(K=257), -2), (dict(T=(1 << 27) + 1), -2),
    (dict(V=(1 << 28) + 1), -2), (dict(dtype=2), -1), (dict(temperature=0.0), -1), (dict(temperature=-2.0), -1),
    (dict(temperature=float("inf")), -1), (dict(temperature=1e-39), -1), (dict(scale=float("nan")), -1),
    (dict(ld_logits=99), -1), (dict(logits=0), -1), (dict(logits=PTR + 1), -1), (dict(t_ids=0), -1),
    (dict(t_logits=0), -1), (dict(t_lse=PTR + 2), -1), (dict(T=0), 0), (dict(T=0, logits=0), 0),
])
def test_distill_refusals(L, kw, want):
    for f in (L.moe_distill, L.moe_distill_backward, L.moe_distill_step):
        assert f(distill(**kw), None) == want


def test_distill_outputs(L):
    assert L.moe_distill(distill(loss=0), None) == -1 and L.moe_distill(distill(lse=0), None) == -1
    assert L.moe_distill_backward(distill(lse=0), None) == -1 and L.moe_distill_backward(distill(weight=0), None) == -1
    assert L.moe_distill_step(distill(dlogits=0), None) == -1
    assert L.moe_distill_step(distill(ld_logits=128, ld_dlogits=100), None) == -1  # in place, another stride


def test_cpu_tensors_are_refused():
    t = torch.ones(4, 8)
    for f in (lambda: moe.block_norm(t, None, None, t[0]), lambda: moe.embed(t, torch.zeros(2, dtype=torch.int64)),
              lambda: moe.distill(t, torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, 1))):
        with pytest.raises(ValueError):
            f()


def test_a_workspace_has_the_bytes_it_names():
    """A broadcast tensor names more elements than it holds."""
    cpu = types.SimpleNamespace(index=-1)  # as a CPU tensor's get_device() says
    one = torch.empty(1, dtype=torch.uint8)
    assert step._ws(0, one, cpu) == (one, 1) and step._ws(0, torch.empty(6), cpu)[1] == 24
    for ws in (one.expand(1 << 20), torch.empty(64, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            step._ws(0, ws, cpu)


def test_autograd_learns_of_writes_into_the_callers_tensors(monkeypatch):
    """(the calls themselves are left out: only the bookkeeping runs here)"""
    for n in ("moe_block_norm", "moe_embed_backward", "moe_distill_backward", "moe_distill_step"):
        monkeypatch.setattr(step, n, lambda *a: None)
    monkeypatch.setattr(step, "moe_embed_workspace_size", lambda a: 256)
    monkeypatch.setattr(step, "_ws", lambda n, ws, dev: (torch.empty(n, dtype=torch.uint8), n))
    r, y, w = torch.ones(4, 8), torch.ones(4, 8), torch.ones(8)
    norm = lambda inplace, y: step._block_norm(None, r, y, None, w, None, 1.0, 1e-6, 0.0, None, inplace)  # noqa: E731
    norm(False, y), norm(True, None)
    assert r._version == 0 and y._version == 0
    assert norm(True, y)[0] is r and r._version == 1 and y._version == 0 and w._version == 0
    table = torch.zeros(5, 8)
    back = lambda t: step._embed_backward(None, torch.zeros(4, dtype=torch.int64), y, 5, 1.0, None, t, None)  # noqa: E731
    assert back(None)._version == 0 and back(table) is table and table._version == 1 and y._version == 0
    z, ids, t, ones = torch.ones(4, 9), torch.zeros(4, 2, dtype=torch.int32), torch.ones(4, 2), torch.ones(4)
    for n, mode in ((0, 2), (2, 3)):
        call = lambda out: step._distill(None, z, ids, t, 1.0, 1.0, None, ones, ones, out, mode)  # noqa: E731
        call(None)
        assert z._version == n
        other = torch.empty(4, 9)
        call(other)
        assert other._version == 1 and z._version == n
        call(z)
        assert z._version == n + 1
        z.add_(0)
    assert ids._version == t._version == ones._version == 0


def test_second_derivatives_raise(monkeypatch):
    """Where another path keeps the graph alive, too: the gradient of a square
    of a gradient would otherwise lack the operator's part without a word."""
    from top_routed_grouped_gb300 import step_layer as m
    monkeypatch.setattr(m, "embed", lambda table, ids, scale, out_dtype: table[ids] * scale)
    monkeypatch.setattr(m, "embed_backward", lambda ids, dout, V, scale, padding_id: torch.zeros(V, dout.shape[1]).index_add_(0, ids, dout * scale))
    monkeypatch.setattr(m, "block_norm", lambda r, y, *a, **k: (r + y, r * y))
    monkeypatch.setattr(m, "block_norm_backward", lambda d, dh, r, y, *a, **k: dict(dr=d + dh, dy=d - dh, dw_post=None, dw_pre=y[0] + 0, dgate=None))
    monkeypatch.setattr(m, "distill", lambda z, *a: (z.sum(1), z.sum(1)))
    monkeypatch.setattr(m, "distill_backward", lambda w, lse, z, *a: w[:, None] * z)
    ids, w = torch.tensor([0, 2]), torch.ones(3)
    for f, shape in ((lambda x: m.EmbedFunction.apply(x, ids, 2.0, None, None), (4, 3)),
                     (lambda x: sum(m.BlockNormFunction.apply(x, 2 * x, None, w, None, 1.0, 1e-6, 0.0, None)), (2, 3)),
                     (lambda x: m.distillation_loss(x, ids[:, None], x.detach()), (2, 3))):
        x = torch.randn(shape, requires_grad=True)
        out = f(x)
        (g,) = torch.autograd.grad(out.square().sum() + x.square().sum(), x, create_graph=True)
        assert g.requires_grad
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.square().sum().backward()


def test_second_derivatives_of_the_layer_raise(monkeypatch):
    from top_routed_grouped_gb300 import layer as m
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    saved = {n: torch.zeros(1) for n in m._ROUTING}
    monkeypatch.setattr(m, "forward", lambda x, *a, **k: dict(saved, y=x * 2, saved={n: torch.zeros(1) for n in m._SAVED}))
    names = ("dw_router", "dw_shared_gate", "dw_gate_up", "dw_down", "dws_gate_up", "dws_down")
    monkeypatch.setattr(m, "backward", lambda f, dy, x, *w, **k: dict({n: v + 0 for n, v in zip(names, w)}, dx=dy * 2))
    x = torch.randn(3, 4, requires_grad=True)
    y = m.MoEFunction.apply(x, *[torch.zeros(2) for _ in names], 1)[0]
    (g,) = torch.autograd.grad(y.square().sum() + x.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.square().sum().backward()


def test_padding_tokens():
    """The module's -1 is the last token, as in torch, not none; one past the
    table is an error."""
    make = lambda p: moe.TokenEmbedding(10, 4, padding_id=p, device="cpu")  # noqa: E731
    assert make(None).padding_id is None and make(3).padding_id == 3 and make(0).padding_id == 0
    assert make(-1).padding_id == 9 and make(-10).padding_id == 0
    for bad in (10, -11):
        with pytest.raises(ValueError):
            make(bad)


def test_kinds_of_gates():
    """A float [T, 1] beside bfloat16 rows of one channel is a token's gate."""
    kind = lambda gate, H, dtype: step._norm_weights(dtype, H, -1, None, None, gate, 5)[0]  # noqa: E731
    ones, b16 = torch.ones(5, 1), torch.bfloat16
    assert kind(ones, 1, b16) == kind(ones, 8, b16) == kind(ones, 8, torch.float32) == 1
    assert kind(ones.to(b16), 1, b16) == kind(ones, 1, torch.float32) == 3
    assert kind(torch.ones(8), 8, torch.float32) == 2 and kind(torch.ones(5, 8), 8, torch.float32) == 3
    with pytest.raises(ValueError):
        kind(ones.to(b16), 8, b16)


def test_a_row_keeps_the_stride_of_its_matrix():
    wide = torch.zeros(6, 12)
    rows = lambda t: step._rows(t, t.shape[0], t.shape[1], torch.float32, -1, "r")  # noqa: E731
    assert rows(wide) == (wide, 0) and rows(wide[2:3])[1] == 0
    assert rows(wide[:, :8])[1] == 12 and rows(wide[2:3, :8])[1] == 12 and rows(wide[2:3, 3:4])[1] == 12
    assert rows(torch.zeros(1, 8))[1] == 0 and rows(torch.zeros(8, 1).t())[1] == 0
    assert rows(torch.zeros(1, 8).expand(1, 8))[1] == 0 and rows(torch.zeros(1, 1).expand(1, 8))[1] == 0
    for t in (wide[2:3, :8], wide[:, :8], wide, torch.zeros(8, 1).t(), wide[:, 5:6]):
        ld = rows(t)[1]
        like = step._like(t, ld, torch.bfloat16)
        assert like.shape == t.shape and rows(like.float())[1] == 0 and like.dtype is torch.bfloat16
        assert step._like(t, ld).dtype is torch.float32
