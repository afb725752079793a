"""C-ABI and Python argument checks of a layer's operators (linear attention, tokens by expert,
dropout) that need no GPU: a host-only context validates every argument before it refuses the launch."""

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "muon.h")
B = pytest.importorskip("matrix_orthogonalising_optimizer_muon_amd.binding")
FAKE = 0x100000  # never dereferenced: host-only contexts launch nothing


@pytest.fixture(scope="module")
def hctx():
    ctx = B.muon_init(-1)
    yield ctx
    B.muon_destroy(ctx)


def test_python_struct_layouts_match_c_compiler(tmp_path):
    structs = {n: getattr(B, n) for n in ("muon_mix", "muon_mix_grads", "muon_experts", "muon_drop")}
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void){"]
    for name, cls in structs.items():
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    for c in ("MUON_MIX_MAX_DIM", "MUON_MAX_EXPERTS", "MUON_MAX_CHOICES"):
        lines.append(f'printf("{c} value %d\\n", {c});')
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c99", str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        name, field, val = line.split()
        if field == "value":
            assert getattr(B, name) == int(val), name
        elif field == "size":
            assert ctypes.sizeof(structs[name]) == int(val), name
        else:
            assert getattr(structs[name], field).offset == int(val), (name, field)
    assert set(structs) <= {n for n in dir(B)} and "muon_dropout" in B.exported_symbols() and "muon_mix_step" in B.exported_symbols()


def mix(**kw):
    d = dict(q=FAKE, k=FAKE, v=FAKE, log_decay=FAKE, state=FAKE, lengths=FAKE, q_strides=(640, 64, 16), k_strides=(320, 32, 16),
             v_strides=(480, 48, 24), batch=2, tokens=10, heads=4, kv_heads=2, dim=16, dim_v=24, scale=0.25, dtype=B.MUON_BF16)
    d.update(kw)
    return B.muon_mix(**d)


def mix_grads(**kw):
    d = dict(d_o=FAKE, do_strides=(960, 96, 24), d_final=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, d_state=FAKE)
    d.update(kw)
    return B.muon_mix_grads(**d)


BAD_SIZES = [dict(batch=-1), dict(batch=(1 << 18) + 1, heads=1, kv_heads=1), dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(heads=0), dict(kv_heads=0),
             dict(kv_heads=3), dict(kv_heads=-2), dict(heads=65538), dict(batch=1 << 17, heads=4), dict(dim=0), dict(dim=257),
             dict(dim_v=0), dict(dim_v=257), dict(dtype=2), dict(dtype=-1)]
BAD_REST = [dict(scale=float("nan")), dict(scale=float("inf")), dict(q_strides=(-1, 64, 16)), dict(k_strides=(0, (1 << 40) + 1, 0)),
            dict(v_strides=(0, 0, -8)), dict(q=None), dict(k=None), dict(v=None), dict(log_decay=None), dict(q=FAKE + 1),
            dict(k=FAKE + 1), dict(v=FAKE + 1), dict(dtype=B.MUON_F32, q=FAKE + 2), dict(state=FAKE + 2), dict(lengths=FAKE + 1),
            dict(log_decay=FAKE + 2)]


def test_mix_forward_validation(hctx):
    big = 1 << 40
    call = lambda m, o=FAKE, last=FAKE, ws=FAKE, n=big: B.muon_mix_forward(hctx, m, o, last, ws, n, None)  # noqa: E731
    assert call(mix()) == B.MUON_ERR_DEVICE
    for ok in [dict(state=None), dict(lengths=None), dict(q_strides=(0, 0, 0)), dict(batch=0, q=None, k=None, v=None, log_decay=None)]:
        assert call(mix(**ok)) == (B.MUON_OK if "batch" in ok else B.MUON_ERR_DEVICE), ok
    assert call(mix(tokens=0, q=None, k=None, v=None), o=None, last=None) == B.MUON_OK
    assert call(mix(tokens=0, q=None, k=None, v=None), o=None) == B.MUON_ERR_DEVICE      # the states are wanted
    for bad in BAD_SIZES + BAD_REST:
        assert call(mix(**bad)) == B.MUON_ERR_ARG, bad
    assert call(None) == B.MUON_ERR_ARG
    assert call(mix(), o=None) == B.MUON_ERR_ARG and call(mix(), o=FAKE + 1) == B.MUON_ERR_ARG
    assert call(mix(), last=FAKE + 2) == B.MUON_ERR_ARG and call(mix(), last=None) == B.MUON_ERR_DEVICE
    assert B.muon_mix_forward(None, mix(), FAKE, FAKE, FAKE, big, None) == B.MUON_ERR_ARG
    # few heads and many tokens need states of segments
    long = mix(tokens=1 << 16, batch=1)
    need = B.muon_mix_workspace_size(hctx, long)
    assert need > 0 and need % 256 == 0
    assert call(long, n=need) == B.MUON_ERR_DEVICE
    for kw in (dict(n=need - 1), dict(ws=None), dict(ws=FAKE + 128)):
        assert call(long, **kw) == B.MUON_ERR_WORKSPACE, kw
    assert B.muon_mix_workspace_size(hctx, mix()) == 0 and call(mix(), ws=None, n=0) == B.MUON_ERR_DEVICE


def test_mix_backward_validation(hctx):
    big = 1 << 40
    call = lambda m, g, ws=FAKE, n=big: B.muon_mix_backward(hctx, m, g, ws, n, None)  # noqa: E731
    assert call(mix(), mix_grads()) == B.MUON_ERR_DEVICE
    none = dict(dq=None, dk=None, dv=None, d_state=None)
    assert call(mix(), mix_grads(**none)) == B.MUON_OK
    for name in none:
        assert call(mix(), mix_grads(**none | {name: FAKE})) == B.MUON_ERR_DEVICE, name
    for bad in BAD_SIZES + BAD_REST:
        assert call(mix(**bad), mix_grads()) == B.MUON_ERR_ARG, bad
    for bad in [dict(d_o=None), dict(d_o=FAKE + 1), dict(do_strides=(0, -1, 0)), dict(dq=FAKE + 1), dict(dk=FAKE + 1), dict(dv=FAKE + 1),
                dict(d_final=FAKE + 2), dict(d_state=FAKE + 2)]:
        assert call(mix(), mix_grads(**bad)) == B.MUON_ERR_ARG, bad
    assert call(mix(), None) == B.MUON_ERR_ARG and call(None, mix_grads()) == B.MUON_ERR_ARG
    # shared heads need their partial gradients
    need = B.muon_mix_workspace_size(hctx, mix(), mix_grads())
    assert need >= 2 * 10 * 4 * (16 + 24) * 4
    assert call(mix(), mix_grads(), n=need - 1) == B.MUON_ERR_WORKSPACE and call(mix(), mix_grads(), n=need) == B.MUON_ERR_DEVICE
    assert B.muon_mix_workspace_size(hctx, mix(kv_heads=4), mix_grads()) == 0
    assert call(mix(tokens=0), mix_grads(d_state=None)) == B.MUON_OK


def test_mix_workspace_size_refuses_what_the_calls_refuse(hctx):
    n = ctypes.c_size_t()
    for bad in BAD_SIZES:
        assert B._lib.muon_mix_workspace_size(hctx, mix(**bad), None, n) == B.MUON_ERR_ARG, bad
    assert B._lib.muon_mix_workspace_size(hctx, mix(), None, None) == B.MUON_ERR_ARG
    assert B._lib.muon_mix_workspace_size(None, mix(), None, n) == B.MUON_ERR_ARG
    # the largest sizes' arithmetic stays within 64 bits
    most = mix(batch=1 << 18, tokens=1 << 24, heads=1, kv_heads=1, dim=256, dim_v=256)
    assert B._lib.muon_mix_workspace_size(hctx, most, mix_grads(), n) == B.MUON_OK
    assert B._lib.muon_mix_workspace_size(hctx, mix(batch=4, tokens=1 << 24, heads=65536, kv_heads=1, dim=256, dim_v=256),
                                          mix_grads(), n) == B.MUON_OK


def test_mix_step_validation(hctx):
    ok = dict(tokens=1, lengths=None)
    call = lambda m, o=FAKE, new=FAKE: B.muon_mix_step(hctx, m, o, new, None)  # noqa: E731
    assert call(mix(**ok)) == B.MUON_ERR_DEVICE
    nbytes = 2 * 4 * 16 * 24 * 4
    assert call(mix(**ok), new=FAKE + nbytes) == B.MUON_ERR_DEVICE and call(mix(**ok), new=FAKE - nbytes) == B.MUON_ERR_DEVICE
    for new in (FAKE + 4, FAKE + nbytes - 4, FAKE - 4, FAKE - nbytes + 4, None, FAKE + 2):
        assert call(mix(**ok), new=new) == B.MUON_ERR_ARG, new
    for bad in [dict(tokens=2), dict(tokens=0), dict(lengths=FAKE), dict(state=None)]:
        assert call(mix(**ok | bad)) == B.MUON_ERR_ARG, bad
    assert call(mix(**ok), o=None) == B.MUON_ERR_ARG and call(mix(**ok), o=FAKE + 1) == B.MUON_ERR_ARG
    assert call(mix(**ok | dict(batch=0)), o=None, new=None) == B.MUON_OK


def choices(**kw):
    d = dict(ids=FAKE, order=FAKE, slots=FAKE, offsets=FAKE, tokens=100, top=3, experts=7, id_dtype=B.MUON_I64, reserved=0)
    d.update(kw)
    return B.muon_experts(**d)


BAD_CHOICES = [dict(tokens=-1), dict(tokens=1 << 24), dict(top=0), dict(top=65), dict(tokens=1 << 20, top=33), dict(experts=0),
               dict(experts=1025), dict(reserved=1)]


def test_expert_plan_validation(hctx):
    call = lambda e, ws=FAKE, n=1 << 30: B.muon_expert_plan(hctx, e, ws, n, None)  # noqa: E731
    assert call(choices()) == B.MUON_ERR_DEVICE and call(choices(id_dtype=B.MUON_I32)) == B.MUON_ERR_DEVICE
    assert call(choices(tokens=0, ids=None, order=None, slots=None)) == B.MUON_ERR_DEVICE    # the offsets are written
    for bad in BAD_CHOICES + [dict(id_dtype=0), dict(ids=None), dict(order=None), dict(slots=None), dict(offsets=None),
                              dict(ids=FAKE + 4), dict(order=FAKE + 2), dict(slots=FAKE + 1), dict(offsets=FAKE + 2)]:
        assert call(choices(**bad)) == B.MUON_ERR_ARG, bad
    assert call(None) == B.MUON_ERR_ARG
    n = ctypes.c_size_t()
    for bad in BAD_CHOICES:
        assert B._lib.muon_expert_plan_workspace_size(hctx, choices(**bad), n) == B.MUON_ERR_ARG, bad
    assert B.muon_expert_plan_workspace_size(hctx, choices()) == 0
    assert B.muon_expert_plan_workspace_size(hctx, choices(tokens=1 << 19)) > 0
    many = choices(tokens=1 << 20, top=32)
    need = B.muon_expert_plan_workspace_size(hctx, many)
    assert need > 0 and need % 256 == 0 and call(many, n=need) == B.MUON_ERR_DEVICE
    for kw in (dict(n=need - 1), dict(ws=None), dict(ws=FAKE + 64)):
        assert call(many, **kw) == B.MUON_ERR_WORKSPACE, kw


def test_expert_rows_validation(hctx):
    F, bf = FAKE, B.MUON_BF16
    dispatch = lambda e=None, x=F, ldx=40, xs=F, lds=40, dim=40, dt=bf: B.muon_expert_dispatch(hctx, e or choices(ids=None, order=None), x, ldx, xs, lds, dim, dt, None)  # noqa: E731,E501
    combine = lambda e=None, ys=F, lds=40, w=F, y=F, ldy=40, dim=40, dt=bf: B.muon_expert_combine(hctx, e or choices(), ys, lds, w, y, ldy, dim, dt, None)  # noqa: E731,E501
    back = lambda e=None, dy=F, ldy=40, ys=F, lds=40, w=F, dys=F, ldd=40, dw=F, dim=40, dt=bf: B.muon_expert_combine_backward(hctx, e or choices(), dy, ldy, ys, lds, w, dys, ldd, dw, dim, dt, None)  # noqa: E731,E501
    for call in (dispatch, combine, back):
        assert call() == B.MUON_ERR_DEVICE
        for bad in BAD_CHOICES + [dict(slots=None), dict(offsets=None), dict(slots=F + 2), dict(offsets=F + 1)]:
            assert call(choices(**bad)) == B.MUON_ERR_ARG, bad
        for kw in (dict(dim=0), dict(dim=(1 << 20) + 1), dict(dim=41), dict(dt=2)):
            assert call(**kw) == B.MUON_ERR_ARG, kw
    empty = choices(tokens=0, slots=None, offsets=None)
    assert dispatch(empty, x=None, xs=None) == combine(empty, ys=None, y=None) == back(empty, dy=None, ys=None) == B.MUON_OK
    for kw in (dict(x=None), dict(xs=None), dict(x=F + 1), dict(xs=F + 1), dict(ldx=39), dict(lds=39), dict(lds=(1 << 36) + 1)):
        assert dispatch(**kw) == B.MUON_ERR_ARG, kw
    for kw in (dict(ys=None), dict(y=None), dict(w=F + 2), dict(lds=39), dict(ldy=39), dict(y=F + 1)):
        assert combine(**kw) == B.MUON_ERR_ARG, kw
    for kw in (dict(dy=None), dict(ys=None), dict(dw=F + 2), dict(w=F + 1), dict(ldy=39), dict(lds=39), dict(ldd=39), dict(dys=F + 1)):
        assert back(**kw) == B.MUON_ERR_ARG, kw
    assert combine(w=None) == B.MUON_ERR_DEVICE
    assert back(ys=None, lds=0, dw=None) == B.MUON_ERR_DEVICE and back(dys=None, ldd=0) == B.MUON_ERR_DEVICE
    assert back(dys=None, dw=None) == B.MUON_OK


def drop(**kw):
    d = dict(x=FAKE, residual=FAKE * 2, out=FAKE * 3, counter=None, ld_x=40, ld_residual=40, ld_out=40, rows=10, cols=40, seed=1,
             offset=2, p=0.1, dtype=B.MUON_BF16)
    d.update(kw)
    return B.muon_drop(**d)


def test_dropout_validation(hctx):
    call = lambda d: B.muon_dropout(hctx, d, None)  # noqa: E731
    for ok in [dict(), dict(residual=None, ld_residual=0), dict(counter=FAKE), dict(p=0.0), dict(p=1.0), dict(out=FAKE),
               dict(out=FAKE * 2), dict(ld_x=100, out=FAKE + 80, ld_out=100), dict(rows=1, ld_x=50, out=FAKE)]:
        assert call(drop(**ok)) == B.MUON_ERR_DEVICE, ok
    assert call(drop(rows=0, x=None, out=None)) == B.MUON_OK
    for bad in [dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=(1 << 34) + 1, ld_x=1 << 35, ld_out=1 << 35),
                dict(rows=1 << 28, cols=65, ld_x=65, ld_out=65, ld_residual=65), dict(p=-0.1), dict(p=1.5), dict(p=float("nan")),
                dict(ld_x=39), dict(ld_out=39), dict(ld_residual=39), dict(ld_x=(1 << 36) + 1), dict(x=None), dict(out=None),
                dict(x=FAKE + 1), dict(out=FAKE + 1), dict(residual=FAKE + 1), dict(counter=FAKE + 4), dict(dtype=2),
                dict(rows=1 << 26, cols=1, ld_x=1 << 35, ld_out=1 << 35, residual=None), dict(out=FAKE + 2), dict(out=FAKE * 2 + 80), dict(out=FAKE, ld_out=80), dict(ld_x=100, out=FAKE + 78, ld_out=100)]:
        assert call(drop(**bad)) == B.MUON_ERR_ARG, bad
    assert call(None) == B.MUON_ERR_ARG and B.muon_dropout(None, drop(), None) == B.MUON_ERR_ARG


def test_python_arguments_off_the_gpu():
    import torch
    from matrix_orthogonalising_optimizer_muon_amd import dropout, experts, mixers
    x = torch.zeros(2, 3, 4, 8)
    with pytest.raises(ValueError, match="not on a GPU"):
        mixers.linear_attention_forward(x, x, x, torch.zeros(4))
    with pytest.raises(ValueError, match="not on a GPU"):
        experts.expert_plan(torch.zeros(3, 2, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="not on a GPU"):
        dropout.dropout(x, 0.1, 3)
    with pytest.raises(ValueError):
        mixers.DecayAttention(8, 3, 4, kv_heads=2)
    with pytest.raises(ValueError):
        experts.RoutedFeedForward(8, 8, 4, 0)
    with pytest.raises(TypeError):
        dropout.Dropout(0.1, seed=0.5)
