"""Host-side checks of what the operators between a layer's products refuse: results
that share a buffer, results over inputs that are laid out otherwise, and what the
binding would leave out.  Made-up addresses: every refused call ends before any
device work."""
import pytest
import torch

from tests.test_layer_cpu import EINVAL, L, codes, gate, gate_grad, heads, heads_grad  # noqa: F401 (L: a fixture)


def test_results_in_one_buffer(L):
    """Two results of a call in one buffer are refused: codes or scales alone too, the queries' and the keys' as well."""
    c = codes(L, ld=112, lds=100)
    for other in (c, codes(L, codes=1 << 24, ld=112, lds=100), codes(L, scales=1 << 24, ld=112, lds=100)):
        one = dict(rows=100)
        for pair in (("q", "gate_q"), ("q", "up_q"), ("gate_q", "up_q")):
            assert gate(L, **one, **dict(zip(pair, (c, other)))) == EINVAL
            assert "same buffer" in L.opt_last_error()
        outs = ("dgate_q", "dup_q", "dgate_t", "dup_t", "y_t")
        for i, a in enumerate(outs):
            for b in outs[:i]:
                assert gate_grad(L, **one, **{a: c, b: other}) == EINVAL
                assert "same buffer" in L.opt_last_error()
        for a in outs[2:]:
            for b in ("gate_q", "up_q"):
                assert gate_grad(L, True, **one, **{b: c, a: other, "up_q" if b == "gate_q" else "gate_q": codes(L, 1 << 25, 112, 1 << 26, 100)}) == EINVAL
                assert "same buffer" in L.opt_last_error()
        assert heads(L, q=dict(codes=c), k=dict(codes=other)) == EINVAL
        assert "same buffer" in L.opt_last_error()
    assert heads(L, q=dict(y=1 << 27), k=dict(y=1 << 27)) == EINVAL
    assert "two y" in L.opt_last_error()
    assert heads_grad(L, q=dict(dx=1 << 27), k=dict(dx=1 << 27)) == EINVAL
    assert "two dx" in L.opt_last_error()


def test_results_over_inputs(L):
    """A result over an input is refused where their strides differ, or where it is the other set's."""
    for p in (4096, 8192):
        assert gate(L, y=p, ldy=101) == EINVAL
        assert "leading dimension" in L.opt_last_error()
    for out, ld in (("dgate", "lddg"), ("dup", "lddu")):
        for p in (4096, 8192, 12288):
            assert gate_grad(L, **{out: p, ld: 101}) == EINVAL
            assert "leading dimension" in L.opt_last_error()
        assert gate_grad(L, True, **{out: 4096, ld: 101}) == EINVAL
        assert "leading dimension" in L.opt_last_error()
    x = 1 << 14
    for kw in (dict(y_token=193), dict(y_token=200, y_head=65), dict(y_token=64, y_head=320)):
        assert heads(L, q=dict(y=x, **kw)) == EINVAL
        assert "strides" in L.opt_last_error()
        assert heads_grad(L, q=dict(dx=x, **{"d" + k.replace("y", "x"): v for k, v in kw.items()})) == EINVAL
        assert "strides" in L.opt_last_error()
    for kw in (dict(q=dict(y=1 << 16)), dict(k=dict(y=x))):
        assert heads(L, **kw) == EINVAL
        assert "other set" in L.opt_last_error()
    for kw in (dict(q=dict(dx=1 << 16)), dict(q=dict(dx=(1 << 16) + (1 << 11))), dict(k=dict(dx=x)), dict(k=dict(dx=x + (1 << 11)))):
        assert heads_grad(L, **kw) == EINVAL
        assert "other set" in L.opt_last_error()


def test_keys_results_need_keys(L, monkeypatch):
    """The binding refuses results of keys that are not given, forward as backward."""
    monkeypatch.setattr(L, "_device", lambda: -1)       # a host tensor's device number
    h = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for kw in (dict(k_out=h), dict(k_codes=L.block_buffers(8, 64, device="cpu"))):
        with pytest.raises(ValueError, match="need k"):
            L.opt_head_norm(h, None, q_out=h, **kw)


def test_rotation_table_of_odd_size(L):
    """A table has rot columns or is refused (an odd rot gave one more)."""
    for rot in (1, 63, -2):
        with pytest.raises(ValueError, match="even"):
            L.rotation_table(9, rot, device="cpu")
    assert L.rotation_table(9, 0, device="cpu").shape == (9, 0)
