"""What a call writes, its kernels do not read through the read-only path: `__ldg` (ld.global.nc) is defined only for
memory that stays as it is while the kernel runs, and the compiler may repeat such a load or move it over a wait."""
import os
import re

from decode_context_attention_gb300 import build


def code(name):
    """The source without comments."""
    text = open(os.path.join(build.CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def read_only_loads(text):
    """The arguments of every __ldg."""
    found = []
    for m in re.finditer(r"__ldg\s*\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        found.append(text[m.end():i - 1])
    return found


def body(text, head):
    """The function whose definition begins with `head`."""
    i = text.index("{", text.index(head))
    depth, j = 1, i + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        j += 1
    return text[i:j]


def test_the_reader_finds_what_it_looks_for():
    assert read_only_loads("x = __ldg(p.a + f(b)) + __ldg (q);") == ["p.a + f(b)", "q"]
    assert body("int f(int a) { if (a) { g(); } }  int h() {}", "int f(") == "{ if (a) { g(); } }"


def test_the_plan_of_the_prefix_attention():
    # written by the plan kernel, which the kernels that read it may overlap
    assert not read_only_loads(body(code("dcp_chunk.cuh"), "Planned load_planned(const int4* at)"))
    for name in sorted(os.listdir(build.CSRC)):
        for x in read_only_loads(code(name)):
            assert not re.search(r"\b(plan|slim|nothing|pos|wo|wl)\b(?!\s*\()", x), (name, x)


def test_the_numbers_of_free_pages():
    # a call may write the new numbers where the old ones were; the table and the starts are written before they are read
    loads = read_only_loads(code("dcp_pages.cu"))
    assert loads
    for x in loads:
        assert not re.search(r"\b(free_count|free_out|missing|query_start|seq_lens|positions|slots|requests)\b", x), x
    text = code("dcp_pages.cu")
    for head in ("void reserve_rank(", "void reserve_rest("):
        assert not any(re.search(r"\bbt\b|\brow\b", x) for x in read_only_loads(body(text, head))), head
