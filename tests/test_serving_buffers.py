"""Buffers that a caller of the serving operators keeps: those of another
call's size are refused before the library, which sees addresses only."""
import pytest
import torch

import dual_scale_solver_b200 as dq
from dual_scale_solver_b200 import serving


@pytest.fixture
def called(monkeypatch):
    """The binding on CPU tensors without the library; the calls it made."""
    from dual_scale_solver_b200 import build
    build.build()
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(serving, "_lib", lambda: Library())
    monkeypatch.setattr(serving, "_device", lambda tensors: 0)
    monkeypatch.setattr(serving, "_call", lambda device, s, fn, *a: calls.append(a) or 0)
    return calls


@pytest.mark.parametrize("name,G,code_row,scales,wide", [("mxfp4", 32, 32, 2, False), ("mxfp8_e4m3", 32, 64, 2, False),
                                                         ("mxfp6_e2m3", 16, 48, 4, False), ("int4_bf16", 64, 32, 1, True)])
def test_norm_outputs_of_another_size(called, name, G, code_row, scales, wide):
    f = dq.format_preset(name, G)
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64)
    st, other = (torch.int16, torch.uint8) if wide else (torch.uint8, torch.int16)
    codes = lambda t, n, dt=torch.uint8: torch.zeros(t, n, dtype=dt)      # noqa: E731
    good = codes(4, code_row), codes(4, scales, st)
    got = dq.add_rmsnorm_quant(x, w, f, codes=good[0], gscales=good[1])
    assert got[0] is good[0] and got[1] is good[1]
    dq.add_rmsnorm_quant(x, w, f, codes=good[0].view(torch.int8).view(-1), gscales=good[1].view(-1))
    dq.add_rmsnorm_quant(x, w, f, codes=good[0])
    dq.add_rmsnorm_quant(x, w, f, gscales=good[1])
    assert len(called) == 4
    bad = [dict(codes=codes(3, code_row)),                      # fewer tokens
           dict(codes=codes(5, code_row)),
           dict(codes=codes(4, code_row // 2)),                 # fewer channels, a narrower code
           dict(codes=codes(4, 2 * code_row)[:, ::2]),
           dict(gscales=codes(3, scales, st)),
           dict(gscales=codes(4, 2 * scales, st)),              # a smaller group
           dict(gscales=codes(4, scales, other)),               # another format's
           dict(gscales=codes(4, 2 * scales, st)[:, ::2])]
    for kw in bad:
        for more in (dict(), dict(codes=good[0]), dict(gscales=good[1])):
            with pytest.raises(ValueError):
                dq.add_rmsnorm_quant(x, w, f, **{**more, **kw})
    with pytest.raises(dq.DqError) as e:                        # a format that is none, buffers or not
        dq.add_rmsnorm_quant(x, w, dq.dq_format(9, 32, 1, 0, 0), codes=good[0], gscales=good[1])
    assert e.value.status == -3 and len(called) == 4
