"""What the kernels' inline assembly has to say to the compiler."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(__file__), "..", "compressed_sparse_attention_decode_gb300", "csrc")


def statements(text):
    for m in re.finditer(r"\basm(?:\s+volatile)?\s*\(", text):
        depth = 0
        for i in range(m.end() - 1, len(text)):
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            if depth == 0:
                yield text[m.start():i + 1]
                break


def test_waits_are_barriers_to_the_compiler_too():
    """what is read after a wait for another warp's writes must not be moved before it: every form of waiting, and every
    arrival that lets others read, clobbers memory"""
    seen = 0
    for path in glob.glob(os.path.join(CSRC, "*")):
        for s in statements(open(path, encoding="utf-8").read()):
            code = " ".join(re.findall(r'"((?:[^"\\]|\\.)*)"', s))
            if re.search(r"try_wait|test_wait|mbarrier\.arrive|bar\.(sync|arrive|red)|barrier\.cluster|griddepcontrol|wait_all|tcgen05\.wait|fence\.proxy", code):
                seen += 1
                assert '"memory"' in s, (os.path.basename(path), s)
    assert seen > 20
