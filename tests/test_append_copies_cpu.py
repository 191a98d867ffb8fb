"""The order of things in the quantising append's source, on the CPU: what a GPU run cannot show without risking what it looks for."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "prefix_cached_kv_gb300", "csrc", "pck_paged_e4m3.cu")


def _kernel():
    """append8_kernel's body without comments."""
    src = re.sub(r"//[^\n]*", "", open(SRC).read())
    at = src.index("{", src.index(" append8_kernel("))
    depth = 0
    for i in range(at, len(src)):
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        if depth == 0:
            return src[at:i + 1]
    raise AssertionError("no end of the kernel")


def _started(body):
    """Where the first asynchronous copy is started: the first call of fetch."""
    m = re.search(r"(?<![\w=] )\bfetch\(\);", body)
    return m.start()


def test_no_return_leaves_copies_in_flight():
    body = _kernel()
    after = body[_started(body):]
    # (a return inside the lambdas of the heads' loop gives a value)
    bare = [m.start() for m in re.finditer(r"\breturn;", after)]
    assert bare, "the kernel leaves rows that are not stored"
    for at in bare:
        assert "cp.async.wait_all;" in after[:at].rsplit("{", 1)[-1], after[max(0, at - 120):at + 7]
    # and the loop over the heads waits for every head that was asked for before it uses it
    assert re.search(r'cp\.async\.wait_group %0;" ::"n"\(DEPTH - 1\)', after)


def test_no_row_is_read_before_it_is_known_to_be_a_sequences():
    """Rows in front of the first sequence and behind the last are neither read nor written: they need not exist."""
    body = _kernel()
    before = body[:_started(body)]
    m = re.search(r"const bool owned = !P\.cu_rows \|\| \(t >= P\.cu_rows\[0\] && t < P\.cu_rows\[P\.B\]\);", before)
    assert m, "a row's copies begin before it is known to be a sequence's"
    assert "A.in" not in before[:m.start()]
    # the copies of the thread's n-th head are those of head next, which starts behind the last head where the row is no one's
    assert re.search(r"int next = owned \? h0 : Ht\b", before) and re.search(r"if \(next < Ht && active\)", before)
