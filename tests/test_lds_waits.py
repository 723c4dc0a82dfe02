"""The barriers of the attention over many rows that leave LDS operations outstanding leave operand
reads outstanding, never a write: on every path to such a barrier the youngest operations, as many as
its wait allows, are reads.  From the device assembly that hipcc writes for the source."""
import os
import re
import subprocess

import pytest

from rotated_bit_linear_amd import build as B

LDS = re.compile(r"^ds_")
WRITE = re.compile(r"^ds_(write|store|add|or|and|max|min|xor|inc|dec|cmpst)")


def kernels(text):
    """name -> list of (label or None, instruction)"""
    out = {}
    for m in re.finditer(r"^(_ZN\w*attn_rows_kernel\w*):.*?^\.Lfunc_end", text, re.S | re.M):
        body = []
        for line in m.group(0).splitlines()[1:]:
            line = line.split(";")[0].strip()
            label = re.match(r"^(\.LBB\w+):", line)
            if label:
                body.append((label.group(1), ""))
            elif line and not line.startswith("."):
                body.append((None, line))
        out[m.group(1)] = body
    return out


def partial_waits(body):
    """(place, operations left) of the waits directly before a barrier that leave some outstanding"""
    for i, (_, ins) in enumerate(body):
        m = re.match(r"s_waitcnt lgkmcnt\((\d+)\)$", ins)
        if m and int(m.group(1)) > 0 and i + 1 < len(body) and body[i + 1][1].startswith("s_barrier"):
            yield i, int(m.group(1))


def condition(body, at, jumped):
    """{(scalar register pair, whether it is zero)} on the way out of a conditional branch: what is
    known from the flag that it tests."""
    m = re.match(r"s_cbranch_vcc(n?z)", body[at][1])
    for i in range(at - 1, -1, -1) if m else ():
        label, ins = body[i]
        c = re.match(r"s_(andn2|and)_b64 vcc, exec, (s\[\d+:\d+\])", ins)
        if c:
            return {(c.group(2), ((c.group(1) == "andn2") == (m.group(1) == "nz")) == jumped)}
        if label or re.search(r"\bvcc\b", ins) or ins.startswith("s_cbranch"):
            break
    return set()


def write_left(body, at, left):
    """A write among the youngest `left` LDS operations of some path that ends before `at`, or None.
    A path that needs a flag which the same path has set the other way is none."""
    jumps = {}
    for i, (_, ins) in enumerate(body):
        m = re.match(r"s_c?branch\w*\s+(\.LBB\w+)", ins)
        if m:
            jumps.setdefault(m.group(1), []).append(i)
    # place, operations passed, write found, flags that have to hold there
    seen, todo = set(), [(at - 1, 0, None, frozenset())]
    while todo:
        i, n, found, want = todo.pop()
        while (i, n, found, want) not in seen:
            seen.add((i, n, found, want))
            if found is not None and not want:
                return found, body[found][1]
            if i < 0 or (n >= left and found is None):
                break
            label, ins = body[i]
            sets = re.match(r"s_\w+ (s\[\d+:\d+\]),(?: (0|-1)$)?", ins)
            if label:
                todo += [(j - 1, n, found, want | condition(body, j, True)) for j in jumps.get(label, [])]
            elif ins.startswith("s_cbranch"):
                want = want | condition(body, i, False)
            elif re.match(r"s_(branch|endpgm|setpc)", ins):
                break                                    # not reached by falling through
            elif sets and not ins.startswith("s_cmp"):
                zero = {w[1] for w in want if w[0] == sets.group(1)}
                if ins.startswith("s_mov_b64") and sets.group(2) and zero - {sets.group(2) == "0"}:
                    break                                # set the other way
                want = frozenset(w for w in want if w[0] != sets.group(1))
            if found is None and re.search(r"lgkmcnt\(0\)", ins):
                break                                    # all older ones are done
            if found is None and LDS.match(ins):
                if WRITE.match(ins):
                    found = i
                n += 1
            i -= 1
    return None


@pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not available")
def test_barriers_leave_reads_only(tmp_path):
    out = str(tmp_path / "attn.s")
    flags = [f for f in B.FLAGS if f != "-fPIC"]
    subprocess.run([B.HIPCC, *flags, "-x", "hip", "--cuda-device-only", "-S", os.path.join(B.CSRC, "attn_kv8.hip"), "-o", out],
                   check=True, capture_output=True)
    found = kernels(open(out).read())
    assert len(found) == 4, list(found)                  # two types, two head sizes
    for name, body in found.items():
        waits = list(partial_waits(body))
        assert waits, name                               # otherwise this test looks for the wrong thing
        for at, left in waits:
            assert write_left(body, at, left) is None, (name, at, left, write_left(body, at, left))
