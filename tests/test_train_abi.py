"""C-ABI and Python argument checks of the training operators (feed-forward block, losses)
that need no GPU: a host-only context validates every argument before it refuses the launch."""

import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "muon.h")
B = pytest.importorskip("matrix_orthogonalising_optimizer_muon_amd.binding")
FAKE = 0x100000  # never dereferenced: host-only contexts launch nothing


@pytest.fixture(scope="module")
def hctx():
    ctx = B.muon_init(-1)
    yield ctx
    B.muon_destroy(ctx)


def test_struct_layouts_match_c_compiler(tmp_path):
    structs = {n: getattr(B, n) for n in ("muon_ffn", "muon_ffn_grads", "muon_logits", "muon_policy", "muon_distill")}
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void){"]
    for name, cls in structs.items():
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    for c in ("MUON_ACT_SILU", "MUON_ACT_GELU_TANH", "MUON_I32", "MUON_I64", "MUON_MAX_TOP"):
        lines.append(f'printf("{c} value %d\\n", {c});')
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c99", str(src), "-o", str(exe)], check=True)
    got = {}
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        name, field, val = line.split()
        got[(name, field)] = int(val)
    for name, cls in structs.items():
        assert got[(name, "size")] == ctypes.sizeof(cls), name
        for f, _ in cls._fields_:
            assert got[(name, f)] == getattr(cls, f).offset, (name, f)
    for (name, field), val in got.items():
        if field == "value":
            assert getattr(B, name) == val, name


def ffn(**kw):
    d = dict(x=FAKE, w_gate=FAKE, w_up=FAKE, w_down=FAKE, ld_x=40, ld_gate=40, ld_up=40, ld_down=72, tokens=10, dim=40,
             hidden=72, dtype=B.MUON_BF16, activation=0)
    d.update(kw)
    return B.muon_ffn(**d)


def grads(**kw):
    d = dict(dy=FAKE, saved=FAKE, dx=FAKE, g_gate=FAKE, g_up=FAKE, g_down=FAKE, ld_dy=40, ld_dx=40, ld_g_gate=40,
             ld_g_up=40, ld_g_down=72, g_dtype=B.MUON_F32, accumulate=0)
    d.update(kw)
    return B.muon_ffn_grads(**d)


BAD_BLOCK = [dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(dim=0), dict(hidden=0), dict(dim=(1 << 20) + 1),
             dict(hidden=(1 << 20) + 1), dict(ld_x=39), dict(ld_gate=39), dict(ld_up=39), dict(ld_down=71),
             dict(ld_x=(1 << 21) + 1), dict(dtype=2), dict(dtype=-1), dict(activation=2), dict(x=None),
             dict(w_gate=None), dict(w_up=None), dict(w_down=None), dict(x=FAKE + 1), dict(w_down=FAKE + 1),
             dict(dtype=B.MUON_F32, x=FAKE + 2)]


def test_ffn_forward_validation(hctx):
    big = 1 << 40
    call = lambda f, y=FAKE, ld=40, saved=None, ws=FAKE, n=big: B.muon_ffn_forward(hctx, f, y, ld, saved, ws, n, None)  # noqa: E731
    assert call(ffn()) == B.MUON_ERR_DEVICE
    assert call(ffn(tokens=0, x=None), y=None) == B.MUON_OK
    for bad in BAD_BLOCK:
        assert call(ffn(**bad)) == B.MUON_ERR_ARG, bad
    assert call(ffn(), y=None) == B.MUON_ERR_ARG
    assert call(ffn(), ld=39) == B.MUON_ERR_ARG
    assert call(ffn(), y=FAKE + 1) == B.MUON_ERR_ARG
    assert call(ffn(), saved=FAKE + 8) == B.MUON_ERR_ARG
    need, saved = B.muon_ffn_workspace_size(hctx, ffn())
    assert need >= 10 * 128 * 2 and saved == 2 * 32 * 128 * 4
    assert call(ffn(), n=need) == B.MUON_ERR_DEVICE
    assert call(ffn(), n=need - 1) == B.MUON_ERR_WORKSPACE
    assert call(ffn(), ws=None) == B.MUON_ERR_WORKSPACE
    assert call(ffn(), ws=FAKE + 128) == B.MUON_ERR_WORKSPACE
    assert B._lib.muon_ffn_forward(None, ffn(), FAKE, 40, None, FAKE, big, None) == B.MUON_ERR_ARG
    assert B._lib.muon_ffn_forward(hctx, None, FAKE, 40, None, FAKE, big, None) == B.MUON_ERR_ARG


def test_ffn_backward_validation(hctx):
    big = 1 << 40
    call = lambda f, g, ws=FAKE, n=big: B.muon_ffn_backward(hctx, f, g, ws, n, None)  # noqa: E731
    assert call(ffn(), grads()) == B.MUON_ERR_DEVICE
    assert call(ffn(), grads(dx=None, g_up=None)) == B.MUON_ERR_DEVICE
    assert call(ffn(), grads(dx=None, ld_dx=0, g_gate=None, ld_g_gate=0)) == B.MUON_ERR_DEVICE
    for bad in BAD_BLOCK:
        assert call(ffn(**bad), grads()) == B.MUON_ERR_ARG, bad
    for bad in [dict(dy=None), dict(saved=None), dict(ld_dy=39), dict(ld_dx=39), dict(ld_g_gate=39), dict(ld_g_up=39),
                dict(ld_g_down=71), dict(g_dtype=2), dict(accumulate=2), dict(dy=FAKE + 1), dict(dx=FAKE + 1),
                dict(g_gate=FAKE + 2), dict(saved=FAKE + 8)]:
        assert call(ffn(), grads(**bad)) == B.MUON_ERR_ARG, bad
    assert B._lib.muon_ffn_backward(hctx, ffn(), None, FAKE, big, None) == B.MUON_ERR_ARG
    need, _ = B.muon_ffn_workspace_size(hctx, ffn(), grads())
    assert call(ffn(), grads(), n=need) == B.MUON_ERR_DEVICE
    assert call(ffn(), grads(), n=need - 1) == B.MUON_ERR_WORKSPACE


def test_ffn_no_tokens_needs_nothing(hctx):
    empty = ffn(tokens=0, x=None)
    assert B.muon_ffn_workspace_size(hctx, empty) == (0, 0)
    assert B.muon_ffn_workspace_size(hctx, empty, grads(dy=None, saved=None)) == (0, 0)
    g = grads(dy=None, saved=None, dx=None)
    assert B.muon_ffn_backward(hctx, empty, g, None, 0, None) == B.MUON_ERR_DEVICE


def test_ffn_workspace_counts_the_copies(hctx):
    """Rows or addresses off 16 bytes are copied: more workspace; null pointers count as aligned."""
    base, _ = B.muon_ffn_workspace_size(hctx, ffn(x=None, w_gate=None, w_up=None, w_down=None))
    assert base == B.muon_ffn_workspace_size(hctx, ffn())[0]
    off, _ = B.muon_ffn_workspace_size(hctx, ffn(w_gate=FAKE + 2))
    odd, _ = B.muon_ffn_workspace_size(hctx, ffn(ld_gate=41))
    assert off == odd >= base + 72 * 40 * 2
    assert B._lib.muon_ffn_workspace_size(hctx, ffn(), None, None, None) == B.MUON_ERR_ARG


def logits(**kw):
    d = dict(logits=FAKE, dlogits=FAKE * 2, weights=None, grad_rows=None, loss=FAKE, lse=FAKE, ld=50, ld_d=50, rows=3,
             vocab=50, temperature=1.0, dtype=B.MUON_BF16, lse_given=0)
    d.update(kw)
    return B.muon_logits(**d)


def policy(**kw):
    d = dict(targets=FAKE, old_logp=FAKE, advantages=FAKE, ref_logp=FAKE, logp=FAKE, clip_low=0.2, clip_high=0.2, kl_coef=0.1)
    d.update(kw)
    return B.muon_policy(**d)


def distill(**kw):
    d = dict(top_logits=FAKE, top_ids=FAKE, top_lse=None, ld_top=4, ld_ids=4, top=4, top_dtype=B.MUON_F32, id_dtype=B.MUON_I64)
    d.update(kw)
    return B.muon_distill(**d)


BAD_LOGITS = [dict(logits=None), dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 28) + 1), dict(ld=49), dict(ld_d=49),
              dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")), dict(temperature=float("inf")),
              dict(temperature=1e-45), dict(temperature=5e-39), dict(dtype=2), dict(lse_given=2), dict(lse_given=1, lse=None), dict(logits=FAKE + 1),
              dict(dlogits=FAKE + 1), dict(dlogits=FAKE, ld_d=51), dict(dtype=B.MUON_F32, logits=FAKE + 2)]


def test_policy_validation(hctx):
    call = lambda l, t, ws=None, n=0: B.muon_policy_loss(hctx, l, t, ws, n, None)  # noqa: E731
    assert call(logits(), policy()) == B.MUON_ERR_DEVICE
    assert call(logits(dlogits=None, ld_d=0), policy(kl_coef=0.0, ref_logp=None)) == B.MUON_ERR_DEVICE
    assert call(logits(rows=0, logits=None), policy(targets=None)) == B.MUON_OK
    for bad in BAD_LOGITS:
        assert call(logits(**bad), policy()) == B.MUON_ERR_ARG, bad
    for bad in [dict(targets=None), dict(old_logp=None), dict(advantages=None), dict(ref_logp=None), dict(clip_low=-0.1),
                dict(clip_low=1.1), dict(clip_high=-0.1), dict(clip_high=float("nan")), dict(kl_coef=float("inf"))]:
        assert call(logits(), policy(**bad)) == B.MUON_ERR_ARG, bad
    assert B._lib.muon_policy_loss(None, logits(), policy(), None, 0, None) == B.MUON_ERR_ARG
    assert B._lib.muon_policy_loss(hctx, None, policy(), None, 0, None) == B.MUON_ERR_ARG
    assert B._lib.muon_policy_loss(hctx, logits(), None, None, 0, None) == B.MUON_ERR_ARG
    few = logits(rows=3, vocab=152064, ld=152064, ld_d=152064)
    need = B.muon_loss_workspace_size(hctx, few)
    assert need > 0 and need % 256 == 0
    assert call(few, policy(), FAKE, need) == B.MUON_ERR_DEVICE
    assert call(few, policy(), FAKE, need - 1) == B.MUON_ERR_WORKSPACE
    assert call(few, policy(), FAKE + 128, need) == B.MUON_ERR_WORKSPACE
    assert call(few, policy()) == B.MUON_ERR_WORKSPACE
    # many rows, short rows, or rows that are not read as a whole need none
    for kw in [dict(rows=200), dict(vocab=4096), dict(dlogits=None, lse_given=1)]:
        assert B.muon_loss_workspace_size(hctx, logits(**dict(dict(rows=3, vocab=152064, ld=152064, ld_d=152064), **kw))) == 0


def test_distill_validation(hctx):
    call = lambda l, t, ws=None, n=0: B.muon_distill_loss(hctx, l, t, ws, n, None)  # noqa: E731
    assert call(logits(), distill()) == B.MUON_ERR_DEVICE
    assert call(logits(rows=0, logits=None), distill(top_logits=None)) == B.MUON_OK
    for bad in BAD_LOGITS:
        assert call(logits(**bad), distill()) == B.MUON_ERR_ARG, bad
    for bad in [dict(top=0), dict(top=B.MUON_MAX_TOP + 1, ld_top=2000, ld_ids=2000), dict(ld_top=3), dict(ld_ids=3),
                dict(top_dtype=2), dict(id_dtype=1), dict(top_logits=None), dict(top_ids=None), dict(top_logits=FAKE + 2),
                dict(top_ids=FAKE + 2)]:
        assert call(logits(), distill(**bad)) == B.MUON_ERR_ARG, bad
    assert B._lib.muon_distill_loss(hctx, logits(), None, None, 0, None) == B.MUON_ERR_ARG
    few = logits(rows=3, vocab=152064, ld=152064, ld_d=152064)
    need = B.muon_loss_workspace_size(hctx, few, 64)
    assert need > B.muon_loss_workspace_size(hctx, few, 4)
    t = distill(top=64, ld_top=64, ld_ids=64)
    assert call(few, t, FAKE, need) == B.MUON_ERR_DEVICE
    assert call(few, t, FAKE, need - 1) == B.MUON_ERR_WORKSPACE
    n = ctypes.c_size_t()
    for l, top in [(None, 0), (few, -1), (few, B.MUON_MAX_TOP + 1), (logits(dtype=3), 0), (logits(vocab=0), 0)]:
        assert B._lib.muon_loss_workspace_size(hctx, l, top, n) == B.MUON_ERR_ARG
    assert B._lib.muon_loss_workspace_size(hctx, few, 0, None) == B.MUON_ERR_ARG


def test_loss_overlaps_and_limits(hctx):
    """A gradient that shares memory with the logits is refused unless it is the logits; columns
    side by side in rows of one stride share none."""
    call = lambda l: (B.muon_policy_loss(hctx, l, policy(), None, 0, None),  # noqa: E731
                      B.muon_distill_loss(hctx, l, distill(), None, 0, None))
    row = 50 * 2
    for kw, ok in [(dict(dlogits=FAKE), True), (dict(dlogits=FAKE + row), False), (dict(dlogits=FAKE - row), False),
                   (dict(dlogits=FAKE + 2), False), (dict(dlogits=FAKE + 3 * row), True), (dict(dlogits=FAKE - 3 * row), True),
                   (dict(dlogits=FAKE + 3 * row - 2), False),
                   (dict(ld=100, ld_d=100, dlogits=FAKE + row), True), (dict(ld=100, ld_d=100, dlogits=FAKE + row - 2), False),
                   (dict(ld=100, ld_d=100, dlogits=FAKE + row + 2), False), (dict(ld=101, ld_d=101, dlogits=FAKE + row + 2), True),
                   (dict(ld=100, ld_d=100, dlogits=FAKE - row), True), (dict(ld=100, ld_d=100, dlogits=FAKE + 3 * row), True),
                   (dict(ld=100, ld_d=99, dlogits=FAKE + row), False), (dict(rows=1, dlogits=FAKE + row), True),
                   (dict(rows=(1 << 24) - 1, dlogits=None), True), (dict(rows=1 << 24, dlogits=None), False),
                   (dict(ld=1 << 36, dlogits=None), True), (dict(ld=(1 << 36) + 1, dlogits=None), False),
                   (dict(ld_d=(1 << 36) + 1, rows=1), False)]:
        assert call(logits(**kw)) == ((B.MUON_ERR_DEVICE if ok else B.MUON_ERR_ARG),) * 2, kw


def test_gradient_buffers_that_overlap():
    from matrix_orthogonalising_optimizer_muon_amd.layers import _overlap, _spans
    t = torch.zeros(6, 8)
    apart = [(t[:3], t[3:]), (t[:, :4], t[:, 4:]), (t[:, 4:], t[:, :3]), (t, torch.zeros(6, 8)), (t[:1, :4], t[:1, 4:])]
    shared = [(t, t), (t[:4], t[3:]), (t[:, :5], t[:, 4:]), (t[:, 4:], t[:, :5]), (t[:, :4], t[1:, 3:]),
              (t[:, 2:4], t.view(12, 4)[:, 1:3])]
    for pairs, want in ((apart, False), (shared, True)):
        for k, (a, b) in enumerate(pairs):
            for p, q in ((a, b), (b, a)):
                x, y = _spans((p, q))
                assert _overlap(x, y) == want, (k, want)
    assert _spans((None, t[:0], t[:, :0])) == []


def test_python_refusals():
    """What the Python functions refuse before the library is called (CPU tensors throughout)."""
    from matrix_orthogonalising_optimizer_muon_amd import layers, losses
    x, w, d = torch.zeros(3, 8), torch.zeros(16, 8), torch.zeros(8, 16)
    with pytest.raises(ValueError, match="not on a GPU"):
        layers.ffn_forward(x, w, w, d)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        layers.ffn_forward(x.half(), w, w, d)
    with pytest.raises(TypeError, match="torch.Tensor"):
        layers.ffn_forward([1.0], w, w, d)
    with pytest.raises(ValueError, match="activation"):
        layers.GatedFeedForward(8, 16, activation="relu")
    with pytest.raises(ValueError, match="not on a GPU"):
        losses.policy_loss(x, torch.zeros(3, dtype=torch.int64), torch.zeros(3), torch.zeros(3))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        losses.distill_loss(x.double(), x, torch.zeros(3, 8, dtype=torch.int64))


def test_operand_checks():
    from matrix_orthogonalising_optimizer_muon_amd.context import matrix, vector
    cpu, f32 = torch.device("cpu"), torch.float32
    t = torch.zeros(4, 6)
    assert matrix(t, "t", (4, 6), f32, cpu) == 6
    assert matrix(torch.zeros(4, 9)[:, :6], "t", (4, 6), f32, cpu) == 9
    assert matrix(torch.zeros(1, 6).expand(1, 6), "t", (1, 6), f32, cpu) == 6
    for bad, kind in [(t.T, ValueError), (t[:1].expand(4, 6), ValueError), (t[:, ::2], ValueError), (t.double(), TypeError),
                      (t[:3], ValueError), (None, TypeError)]:
        with pytest.raises(kind):
            matrix(bad, "t", (4, 6), f32, cpu)
    with pytest.raises(ValueError, match="unit column stride"):
        matrix(torch.zeros(4, 12)[:, ::2], "t", (4, 6), f32, cpu)
    for bad, kind in [(torch.zeros(5), ValueError), (torch.zeros(8)[::2], ValueError), (torch.zeros(4).double(), TypeError),
                      (3, TypeError)]:
        with pytest.raises(kind):
            vector(bad, "v", 4, f32, cpu)
