"""The plain and the 64-bit forms of the operators in perf/operators.py, on
the CPU: they agree with each other and with the references of the tests.
They run in a child process: torch's threads, once started, would hang the
forked workers of other tests."""
import os
import subprocess
import sys
import types

import numpy as np
import pytest

import mx_reference as ref

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def operators():
    """The module with its tensors on the CPU."""
    with open(os.path.join(ROOT, "perf", "operators.py")) as f:
        text = f.read()
    m = types.ModuleType("operators_on_cpu")
    exec(compile(text.replace('"cuda"', '"cpu"'), "operators.py", "exec"), m.__dict__)
    return m


@pytest.mark.parametrize("top", (1, 2, 8))
def test_distill_rows_without_entries(top):
    code = (f"import sys; sys.path[:0] = [{ROOT!r}, {HERE!r}]; import test_operators_plain_host as t; "
            f"[t.rows_without_entries({top}, lse, hard) for lse in (False, True) "
            f"for hard in (0.0, 0.3)]; print('BODY_OK')")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "BODY_OK" in r.stdout, r.stdout + r.stderr


def rows_without_entries(top, lse, hard):
    """At top 1 every sixteenth row has no entry of the teacher: its KL is 0
    and only the label's term is left.  The plain form is off by fp32's error:
    sums of 500 terms, exponentials and a few products, 1e-5 relative to the
    row's largest value is over ten times that."""
    ops = operators()
    case = dict(op="distill", rows=34, vocab=500, ld=512, top=top, x="f32", t="f32", idx=64,
                tau=2.0, hard=hard, log2_scale=8, lse=lse)
    st = ops.prepare(case, 3)
    empty = (st["idx"] < 0).all(1).numpy()
    assert empty.any() == (top == 1)
    loss, grad, flag = ops.run(st)
    loss64, grad64, flag64 = ops.exact(case, 3)
    want_l, want_g = ref.distill(
        st["logits"].double().numpy(), st["idx"].numpy(), st["top"].double().numpy(), 2.0,
        1.0 - hard, hard, st["labels"].numpy() if hard else None, st["weight"].double().numpy(),
        st["lse"].double().numpy() if lse else None, 8)
    assert flag.item() == 0 and flag64.item() == 0
    for got in (grad.double().numpy(), grad64.numpy()):
        assert np.isfinite(got).all()
        assert (np.abs(got - want_g) <= 1e-5 * np.abs(want_g).max(1, keepdims=True)).all()
    for got in (loss.double().numpy(), loss64.numpy()):
        assert (np.abs(got - want_l) <= 1e-5 * np.maximum(np.abs(want_l), want_l.max())).all()
    if top == 1 and not hard:
        assert (grad.numpy()[empty] == 0).all() and (loss.numpy()[empty] == 0).all()
