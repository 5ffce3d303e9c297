"""Sizes (M, N, K) of the gated linear layer that reach each kernel of its large products, with cut tiles, cut last stages of
K and at least five stages each.  The key: tiles, LDS slots, whether K is split over workgroups, and whether workgroups take
more than one piece of work.  tests/test_gated_plan_host.py holds them to the library's plan."""

FORWARD = {
    ("128", 4, False, False): (71, 41, 264),
    ("128", 4, True, False): (71, 42, 904),
    ("128", 2, False, False): (16394, 68, 280),
    ("128", 2, False, True): (13725, 522, 272),
    ("128", 2, True, False): (5538, 65, 4896),
    ("128", 2, True, True): (10891, 129, 6560),
    ("256", 2, False, False): (533, 6672, 272),
    ("256", 2, False, True): (15105, 776, 264),
    ("256", 2, True, False): (147, 8245, 3936),
    ("256", 2, True, True): (518, 6659, 7344),
}
# of dx = [dg | du] [w_gate; w_up]: the second operand lies down, K has two halves
DX = {
    ("128", 4, False, False): (66, 136, 40),
    ("128", 4, True, False): (67, 901, 40),
    ("128", 2, False, False): (11651, 130, 272),
    ("128", 2, False, True): (13254, 131, 1104),
    ("128", 2, True, False): (11753, 1552, 40),
    ("192", 2, False, False): (11448, 129, 656),
    ("192", 2, False, True): (7195, 129, 2224),
    ("192", 2, True, False): (8195, 2883, 136),
    ("192", 2, True, True): (11403, 6982, 264),
    ("256", 2, False, False): (8235, 129, 1360),
    ("256", 2, False, True): (3093, 129, 7816),
    ("256", 2, True, False): (8462, 7705, 208),
}
# of [dw_gate; dw_up] = [dg | du]^T x: both operands lie down
DW = {
    ("128", 4, False, False): (267, 40, 40),
    ("128", 4, True, False): (904, 40, 40),
    ("128", 2, False, False): (286, 8238, 136),
    ("128", 2, False, True): (274, 6621, 1056),
    ("128", 2, True, False): (2829, 6077, 40),
    ("192", 2, False, False): (264, 8249, 392),
    ("192", 2, False, True): (263, 8253, 920),
    ("192", 2, True, False): (2771, 8253, 136),
    ("192", 2, True, True): (14615, 5589, 264),
    ("256", 2, False, False): (267, 6867, 776),
    ("256", 2, False, True): (259, 7596, 1568),
    ("256", 2, True, False): (5293, 8294, 200),
}
# K no multiple of 8: operands copied to aligned rows, large tiles behind
PADDED = {"forward": (533, 6672, 271), "dx": (8235, 129, 1361), "dw": (267, 6867, 775)}
