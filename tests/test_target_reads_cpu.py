"""Where domino_sample reads 16 bytes of logits at once, by reading its source: what lies beside a row is not the caller's to
be read, and no result shows it."""
import re

from tests.test_target_waits_cpu import part, source


def test_logits_are_read_whole_only_inside_the_slice():
    text = source("sample.cu")
    reads = [line for line in text.splitlines() if re.search(r"__ldc[gs]\((slice\.)?from\b", line)]
    assert len(reads) == 3
    for line in reads:  # by Slice::read, or in a loop over the whole units
        assert re.search(r"\bread<", line) or "< end)" in line, line
    assert "const int end = slice.whole0 + slice.wholes;" in text
    read = part(text, "void read(int q0, Get get", "template <typename F>")
    fast, slow = read.split("} else {")
    assert "wholes > kSpan && (unsigned)(q0 - whole0) < (unsigned)(wholes - kSpan)" in fast
    assert re.search(r"if \(kShared \? q < units : whole\(q\)\) x\[j\] = get\(q\);", slow) and slow.count("get(q") == 1


def test_whole_units_lie_inside_the_slice():
    """The constructor's arithmetic for every begin, end and alignment: unit q is whole exactly if all its elements are in."""
    for vec in (4, 8):
        for skew in range(vec):
            for n in range(0, 3 * vec + 2):
                units = (skew + n + vec - 1) // vec if n else 0
                whole0 = 1 if skew else 0
                wholes = max(0, (skew + n) // vec - whole0)
                for q in range(units + 2):
                    inside = all(skew <= q * vec + e < skew + n for e in range(vec))
                    assert inside == (whole0 <= q < whole0 + wholes), (vec, skew, n, q)
                # A batch of three units, two apart, that passes the test has no other units.
                for q0 in range(units + 2):
                    span = 2 * 2
                    if wholes > span and 0 <= q0 - whole0 < wholes - span:
                        assert all(whole0 <= q0 + 2 * j < whole0 + wholes for j in range(3))


def test_changing_logits_cannot_lead_past_shared_memory():
    """The passes over a slice read it again: a logit that has risen above the maximum, or more keys than were counted, must
    not become an index outside the histogram or the list."""
    text = source("sample.cu")
    bins = part(text, "int bin(float d) const {", "}")
    assert "__float2uint_rz(b)" in bins  # saturates at 0
    join = part(text, "static __device__ __forceinline__ void join(", "cluster_sync();")
    assert "x < min(s.n_local, kList - base)" in join
    collect = part(text, "collect(Smem& s, const S& slice", "return sum;")
    assert "if (at < kList) s.list[at]" in collect
    assert "v.key[j] = x < n ? s.list[x] : 0;" in text and "kPer = kList / kThr" in text
