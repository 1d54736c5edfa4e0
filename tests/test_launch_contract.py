"""What the header tells a caller who launches kernels of his own behind a call:
no call that it excuses from the wait launches programmatically (no GPU needed:
the header's words against the sources)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAMMATIC = re.compile(r"launch_pdl\(|ProgrammaticStreamSerialization")


def contract():
    with open(os.path.join(ROOT, "include", "ep.h")) as f:
        text = re.sub(r"\n \* ?", "\n", f.read())
    return text[text.index("programmatic stream serialisation"):text.index("bf16 tensors are passed")]


def body(text, name):
    """The definition of a function at the start of a line, to its closing brace."""
    m = re.search(r"^[\w ]+[ *]%s\([^;{]*\) \{\n(.*?)^\}" % name, text, re.M | re.S)
    return m and m.group(1)


def launchers():
    """Entry point -> the launchers that it calls."""
    sources = ""
    for path in sorted(glob.glob(os.path.join(ROOT, "combine_ep_layout_02_gb300", "csrc", "*.cu"))):
        with open(path) as f:
            sources += f.read() + "\n"
    with open(os.path.join(ROOT, "include", "ep.h")) as f:
        names = re.findall(r"EP_API int (ep_\w+)\(", f.read())
    calls = {n: sorted(set(re.findall(r"\bep::(launch_\w+)\(", body(sources, n) or ""))) for n in names}
    programmatic = {l: bool(PROGRAMMATIC.search(body(sources, l) or "")) for l in {l for c in calls.values() for l in c}}
    return calls, programmatic


def test_sources_are_read():
    calls, programmatic = launchers()
    assert calls["ep_linear"] == ["launch_linear_few", "launch_linear_finish", "launch_product"]
    assert not programmatic["launch_product"] and programmatic["launch_linear_finish"]
    assert calls["ep_linear_backward"] == ["launch_act_backward", "launch_product", "launch_weight_finish"]
    assert programmatic["launch_weight_finish"] and not programmatic["launch_act_backward"]


def test_no_call_is_excused_whose_last_kernel_starts_its_successor_early():
    calls, programmatic = launchers()
    excused = re.findall(r"[^.:]*\bare ordinary launches[^.]*", contract())
    for sentence in excused:
        for name in re.findall(r"\bep_\w+", sentence):
            assert not any(programmatic[l] for l in calls[name]), (name, calls[name])


def test_the_wait_is_asked_for_after_every_call():
    assert re.search(r"must wait on the grid\s+dependency \([^)]*\)[^.]*after every call", contract())
